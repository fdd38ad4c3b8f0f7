"""Calls over many tensors that only the host decides: the lifetime of a table's object
and refusals (no GPU: a refused call, and one over a table without elements, ends before
anything is enqueued)."""
import copy
import gc

import pytest

import fsdp_sharded_optimizer_zs_amd as zs
from test_formats_cpu import lib  # noqa: F401  (builds the library if it is not there)

HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)


def test_a_copied_table_outlives_the_first(lib):  # noqa: F811
    """A shallow copy shares the library's object, which lives until both are gone; a deep
    copy, whose tensors would be others than the object describes, is refused."""
    first = zs.MultiTable([], [], [], [])
    second = copy.copy(first)
    with pytest.raises((ValueError, TypeError)):
        copy.deepcopy(first)
    del first
    gc.collect()
    zs.zs_adamw_multi(second, HP)
