"""What the bindings of the windowed, tree and commit calls take and refuse (CPU: the
library is not reached, tensors are stand-ins)."""
import types

import pytest
import torch

import moe_gqa_query_b200 as gq
from moe_gqa_query_b200 import _lib


def test_binding_takes_device_pointers_for_lengths_too():
    assert _lib._lens(4096, "cache_len", 3, 0) == 4096
    assert _lib._lens(None, "tree_len", 3, 0, True) is None
