"""Tests that pass made-up device addresses (test code).

The C ABI's refusals come before any HIP call, so their tests hand the library
addresses that nothing is mapped at, and count on the launch of a call that is
accepted to fail for want of a GPU. Where there is a GPU such a launch would
run on them: those tests are for machines without one.
"""
import types

import pytest
import torch

LOW, HIGH = 1 << 40, 1 << 47  # what the tests make up; above them are keys and seeds


def _is_address(v):
    if isinstance(v, (list, tuple)):
        return any(_is_address(e) for e in v)
    return isinstance(v, int) and LOW <= v < HIGH


def used_by(fn) -> bool:
    """Whether `fn`, a function nested in it or a helper of its module that it
    names holds or reads such an address."""
    seen, todo = set(), [fn.__code__]
    while todo:
        code = todo.pop()
        if code in seen:
            continue
        seen.add(code)
        if any(_is_address(c) for c in code.co_consts):
            return True
        todo += [c for c in code.co_consts if isinstance(c, types.CodeType)]
        for v in (fn.__globals__.get(n) for n in code.co_names):
            if _is_address(v) or (isinstance(v, types.FunctionType) and any(map(_is_address, v.__defaults__ or ()))):
                return True
            if isinstance(v, types.FunctionType) and v.__module__ == fn.__module__:
                todo.append(v.__code__)
    return False


def skip_where_a_gpu_is(items):
    if torch.cuda.device_count() == 0:
        return
    mark = pytest.mark.skip(reason="made-up device addresses: for machines without a GPU")
    for item in items:
        if isinstance(getattr(item, "function", None), types.FunctionType) and used_by(item.function):
            item.add_marker(mark)
