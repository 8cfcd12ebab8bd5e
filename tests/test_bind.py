"""The native argument check of the binding against the Python one (CPU tensors: device -1)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import w4a16_routed_expert_moe_amd as moe

L = moe._lib


class Away(torch.Tensor):
    def get_device(self):
        return 1


@pytest.fixture
def at():
    L.lib()
    assert L._at is not L._checked  # the native one is in use
    return L._at


def test_passes_what_python_passes(at):
    seen = []
    from w4a16_routed_expert_moe_amd import _bind
    _bind.set_checked(lambda *a: seen.append(a) or 7)
    try:
        for dtype in (torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8):
            t = torch.zeros((4, 6), dtype=dtype)
            assert at(-1, t, "t", dtype, 24) == t.data_ptr() and at(-1, t, "t", dtype, 0, True) == t.data_ptr()
            assert at(-1, t[1:], "t", dtype, 18) == t.data_ptr() + 6 * t.element_size()
        assert not seen
        e = torch.zeros(0)
        assert at(-1, e, "e", torch.float32, 0) == 0 and not seen
        t = torch.zeros((4, 6))
        for args in ((0, t, "t", torch.float32, 24), (-1, t, "t", torch.float32, 25), (-1, t, "t", torch.int32, 24),
                     (-1, t[:, 1:], "t", torch.float32, 1), (-1, t.t(), "t", torch.float32, 24),
                     (-1, None, "t", torch.float32, 24, True), (-1, t.numpy(), "t", torch.float32, 24),
                     (-1, t.as_subclass(Away), "t", torch.float32, 24), (-1, t, "t", "float32", 24),
                     (-1, t.to_sparse(), "t", torch.float32, 1)):
            del seen[:]
            assert at(*args) == 7 and len(seen) == 1 and all(a is b for a, b in zip(seen[0], args)), args
    finally:
        _bind.set_checked(L._checked)


def test_errors_are_those_of_the_python_check(at):
    t = torch.zeros(8)
    for args in ((-1, None, "x", torch.float32, 1), (0, t, "x", torch.float32, 1), (-1, t, "x", torch.int8, 1),
                 (-1, t, "x", torch.float32, 9), (-1, 3, "x", torch.float32, 9)):
        with pytest.raises(ValueError, match="x "):
            at(*args)
    assert at(-1, None, "x", torch.float32, 1, True) is None
    with pytest.raises(TypeError):
        at(-1, t)
    with pytest.raises(TypeError):
        at("0", t, "x", torch.float32, 1)
    with pytest.raises((OverflowError, ValueError)):
        at(-1, t, "x", torch.float32, 1 << 80)


def test_a_tensor_without_memory_is_an_error(at):
    t = torch.zeros((3, 8))
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.vmap(lambda row: row + at(-1, row, "row", torch.float32, 8))(t)
    with pytest.raises((RuntimeError, ValueError)):
        at(0, torch.zeros(8, device="meta"), "x", torch.float32, 8)


def test_a_copy_on_write_tensor_gets_memory_of_its_own(at):
    """The address may be written through: it is not the one that the other tensor still reads."""
    for whose in ("clone", "origin"):
        origin = torch.arange(8, dtype=torch.float32)
        clone = torch._lazy_clone(origin)
        written, other = (clone, origin) if whose == "clone" else (origin, clone)
        p = at(-1, written, "out", torch.float32, 8)
        ctypes.memset(p, 0, 32)
        assert p == written.data_ptr() != other.data_ptr()
        assert torch.equal(other, torch.arange(8, dtype=torch.float32)) and not written.any(), whose


@pytest.mark.parametrize("how", ["of another torch", "without a version", "not loadable"])
def test_native_checks_of_another_build_are_not_used(how):
    """A _bind.so that was built for another torch reads tensors at the wrong offsets: the Python checks take its place."""
    program = """
import sys, types, warnings
import torch
import w4a16_routed_expert_moe_amd as moe
name = "w4a16_routed_expert_moe_amd._bind"
other = types.ModuleType(name)
other.at = other.set_checked = lambda *a: sys.exit("the other build's check was used")
other.built_for = "Python 3.10, torch 1.0"
how = sys.argv[1]
if how == "without a version":
    del other.built_for
sys.modules[name] = None if how == "not loadable" else other
moe._bind = other
if how == "not loadable":
    del moe._bind
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    moe._lib.lib()
assert moe._lib._at is moe._lib._checked
assert any("rebuild" in str(w.message) for w in seen), seen
t = torch.zeros(8)
assert moe._lib._at(-1, t, "t", torch.float32, 8) == t.data_ptr()
"""
    r = subprocess.run([sys.executable, "-c", program, how], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
