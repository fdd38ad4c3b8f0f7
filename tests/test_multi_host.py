"""Calls over many tensors that only the host decides: the lifetime of a table's object
and refusals (no GPU: a refused call, and one over a table without elements, ends before
anything is enqueued)."""
import copy
import ctypes
import gc

import pytest

import fsdp_sharded_optimizer_zs_amd as zs
from test_formats_cpu import (A, STEP, entry, hp, lib, make,  # noqa: F401  (fixtures)
                              no_gpu)

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


@pytest.mark.parametrize("state", (zs.ZS_STATE_F32, zs.ZS_STATE_8BIT))
def test_the_step_refuses_an_image_inside_what_it_writes(lib, no_gpu, state):  # noqa: F811
    """Two tensors of 1000 and 5000 elements: an image of 3 chunks of 80 bytes."""
    h = make(lib, [entry(0, 1000, state), entry(1, 5000, state)], state=state)
    es = 4 if state == zs.ZS_STATE_F32 else 1
    inside = [A, A + 3984, A + STEP, A + 2 * STEP + 1000 * es - 8, A + 3 * STEP + 1984,
              A + 16 * STEP - 224, A + 16 * STEP + 19984]
    if state == zs.ZS_STATE_8BIT:
        inside += [A + 5 * STEP - 224, A + 21 * STEP + 16, A + 22 * STEP]
    for at in inside:
        st = lib.zs_adamw_multi(h, at // 16 * 16, ctypes.byref(hp()), None, None, None)
        assert st == zs.ZS_EALIAS, hex(at - A)
        assert "image" in zs.zs_last_error()


@pytest.mark.parametrize("state", (zs.ZS_STATE_NONE, zs.ZS_STATE_F32))
def test_the_norm_refuses_outputs_inside_the_image(lib, no_gpu, state):  # noqa: F811
    h = make(lib, [entry(0, 1000, state), entry(1, 5000, state)], state=state)
    img, sums, nc, ws = A + 12 * STEP, A + 13 * STEP, A + 14 * STEP, A + 15 * STEP
    call = lambda **kw: lib.zs_grad_norm(h, img, 1.0, kw.get("sums", sums), kw.get("nc", nc),
                                         kw.get("ws", ws), None)
    for bad in (dict(sums=img), dict(sums=img + 232), dict(nc=img + 236), dict(nc=img - 4),
                dict(ws=img + 224), dict(ws=img - zs.ZS_NORM_WORKSPACE + 16)):
        assert call(**bad) == zs.ZS_EALIAS, bad
        assert "image" in zs.zs_last_error()
