"""Host side of the page tables' bookkeeping and of the positions of several
axes: argument structs, axis tables and refusals.  No GPU calls: every
refusal happens before anything is enqueued."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = ctypes.CDLL(bgg.LIB_PATH)
NULL, FORMAT, SHAPE, BUFFER, DESC = 1, 2, 3, 6, 7
P = 1 << 20  # stands for a device pointer; no refused call touches it


def describe(type="f16", pages=10, page_size=16, kv_heads=2, head_dim=64):
    return bgg.bgg_cache_describe(type, pages, page_size, kv_heads, head_dim)


def test_argument_structs_have_the_header_layout(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "bgg.h"\n#include <stdio.h>\n#define O(s, f) (int)offsetof(s, f)\n'
                   'int main(void){printf("%d %d %d %d %d %d\\n",(int)sizeof(bgg_rotary_axes_args),'
                   '(int)sizeof(bgg_assign_args),O(bgg_rotary_axes_args,axis_of_pair_dev),'
                   'O(bgg_assign_args,page_table_dev),O(bgg_assign_args,free_capacity),O(bgg_assign_args,slots_dev));'
                   'return 0;}\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [bgg._ROTARY_AXES_ARGS.size, bgg._ASSIGN_ARGS.size, 16, 40, 72, 128]


# --- axis tables -------------------------------------------------------------
def test_axes_in_blocks():
    assert bgg.bgg_rotary_axes([2, 3, 1]).tolist() == [0, 0, 1, 1, 1, 2]
    assert bgg.bgg_rotary_axes([0, 3, 0, 1]).tolist() == [1, 1, 1, 3]
    assert bgg.bgg_rotary_axes([128]).tolist() == [0] * 128


def test_axes_in_turn():
    assert bgg.bgg_rotary_axes([3, 2, 2], "cyclic").tolist() == [0, 1, 2, 0, 1, 2, 0]
    # axis 0 has what the others leave: 24 + 20 + 20 pairs
    got = bgg.bgg_rotary_axes([24, 20, 20], "cyclic")
    want = [i % 3 if i < 60 else 0 for i in range(64)]
    assert got.tolist() == want and np.bincount(got).tolist() == [24, 20, 20]
    assert bgg.bgg_rotary_axes([5, 0, 1], "cyclic").tolist() == [0, 0, 2, 0, 0, 0]
    assert bgg.bgg_rotary_axes([3], "cyclic").tolist() == [0, 0, 0]


@pytest.mark.parametrize("sections,arrangement,status", [
    ([1, 1], 2, FORMAT), ([1, 1], -1, FORMAT), ([], 0, SHAPE), ([1] * 5, 0, SHAPE), ([1, -1], 0, SHAPE), ([0, 0], 0, SHAPE),
    ([128, 1], 0, SHAPE), ([129], 0, SHAPE), ([64, 65], 1, SHAPE), ([1 << 62, 1 << 62], 0, SHAPE),
    # the last pair of axis 1 (of axis 2) would lie past the end
    ([1, 2], 1, SHAPE), ([10, 10, 11], 1, SHAPE), ([0, 1], 1, SHAPE)])
def test_axes_refusals(sections, arrangement, status):
    with pytest.raises(bgg.BggError) as e:
        bgg.bgg_rotary_axes(sections, arrangement)
    assert e.value.status == status


def test_axes_null():
    out = (ctypes.c_uint8 * 128)()
    assert LIB.bgg_rotary_axes(None, ctypes.c_int64(1), 0, out) == NULL
    assert LIB.bgg_rotary_axes((ctypes.c_int64 * 1)(1), ctypes.c_int64(1), 0, None) == NULL


# --- refusals of the device calls ----------------------------------------------
ROTARY = dict(type=1, layout=0, rotary_dim=64, tokens=3, q_heads=4, q=P, q_out=P, k=P, v=P, qs=256, qos=256, ks=128,
              vs=128, positions=P, slots=P, freqs=P, magnitude=1.0, reserved=0, kc=P, vc=P, ksc=0, vsc=0)
AXES = dict(axes=3, stride=3, of=P)
ASSIGN = dict(batch=2, rows=5, lengths=P, counts=P, shared=P, table=P, width=4, stride=4, free=P, capacity=10, count=P,
              lengths_out=P, count_out=P, past=P, starts=P, positions=P, slots=P)


def axes(desc, rotary={}, **change):
    a = dict(AXES, **change)
    return LIB.bgg_rotary_append_axes(ctypes.byref(desc), bgg._ROTARY_ARGS.pack(*dict(ROTARY, **rotary).values()),
                                      bgg._ROTARY_AXES_ARGS.pack(*a.values()), None)


def assign(desc, **change):
    a = dict(ASSIGN, **change)
    return LIB.bgg_cache_assign(ctypes.byref(desc) if desc is not None else None, bgg._ASSIGN_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(axes=-1), SHAPE), (dict(stride=2), SHAPE), (dict(stride=-3), SHAPE),
    (dict(stride=1 << 41), SHAPE), (dict(of=0), NULL), (dict(rotary=dict(rotary_dim=66)), SHAPE),
    (dict(rotary=dict(positions=0)), NULL), (dict(rotary=dict(positions=P + 2)), BUFFER),
    (dict(rotary=dict(tokens=-1)), SHAPE), (dict(rotary=dict(layout=2)), FORMAT)])
def test_rotary_axes_refusals(change, status):
    assert axes(describe(), **change) == status
    assert "bgg_rotary_append_axes" in bgg.bgg_last_error() or status == 0


def test_rotary_axes_null_and_no_tokens():
    d = describe()
    assert LIB.bgg_rotary_append_axes(ctypes.byref(d), bgg._ROTARY_ARGS.pack(*ROTARY.values()), None, None) == NULL
    assert LIB.bgg_rotary_append_axes(ctypes.byref(d), None, bgg._ROTARY_AXES_ARGS.pack(*AXES.values()), None) == NULL
    assert axes(d, rotary=dict(tokens=0)) == 0
    assert axes(d, rotary=dict(tokens=0), stride=0) == 0


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), SHAPE), (dict(batch=4097), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 23) + 1), SHAPE),
    (dict(width=0), SHAPE), (dict(width=1 << 27, stride=1 << 27), SHAPE), (dict(width=-1), SHAPE),
    (dict(batch=4096, width=(1 << 19) + 1, stride=1 << 20), SHAPE), (dict(stride=3), SHAPE), (dict(stride=1 << 41), SHAPE),
    (dict(capacity=0), SHAPE), (dict(capacity=1 << 31), SHAPE), (dict(capacity=-1), SHAPE),
    (dict(lengths=0), NULL), (dict(counts=0), NULL), (dict(table=0), NULL), (dict(free=0), NULL), (dict(count=0), NULL),
    (dict(lengths_out=0), NULL), (dict(count_out=0), NULL), (dict(past=0), NULL), (dict(starts=0), NULL),
    (dict(positions=0), NULL), (dict(slots=0), NULL), (dict(batch=0, starts=0), NULL), (dict(batch=0, free=0), NULL),
    (dict(lengths=P + 2), BUFFER), (dict(counts=P + 1), BUFFER), (dict(shared=P + 2), BUFFER), (dict(table=P + 2), BUFFER),
    (dict(free=P + 3), BUFFER), (dict(count=P + 2), BUFFER), (dict(lengths_out=P + 2), BUFFER),
    (dict(count_out=P + 2), BUFFER), (dict(past=P + 2), BUFFER), (dict(starts=P + 2), BUFFER),
    (dict(positions=P + 2), BUFFER), (dict(slots=P + 4), BUFFER)])
def test_assign_refusals(change, status):
    assert assign(describe(), **change) == status


def test_assign_descriptor():
    assert assign(None) == NULL
    d = describe()
    assert LIB.bgg_cache_assign(ctypes.byref(d), None, None) == NULL
    d.total_bytes += 1
    assert assign(d) == DESC


# --- attention of groups ---------------------------------------------------------
ATTENTION = dict(type=1, scale=0.1, batch=2, q_heads=4, window=0, q=P, out=P, qs=256, os=256, lse=P, kc=P, vc=P, ksc=0,
                 vsc=0, table=P, width=4, stride=4, lengths=P, ws=P, wsb=1 << 40)
SHARED = dict(groups=1, starts=P, shared=P)


def shared(desc, attention={}, **change):
    return LIB.bgg_shared_attention(ctypes.byref(desc), bgg._ATTENTION_ARGS.pack(*dict(ATTENTION, **attention).values()),
                                    bgg._SHARED_ARGS.pack(*dict(SHARED, **change).values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(groups=-1), SHAPE), (dict(groups=3), SHAPE), (dict(groups=1 << 40), SHAPE), (dict(starts=0), NULL),
    (dict(shared=0), NULL), (dict(starts=P + 2), BUFFER), (dict(shared=P + 1), BUFFER),
    (dict(attention=dict(q_heads=3)), SHAPE), (dict(attention=dict(type=2)), FORMAT), (dict(attention=dict(q=0)), NULL),
    (dict(attention=dict(wsb=1 << 16)), BUFFER), (dict(attention=dict(ws=P + 8)), BUFFER),
    (dict(groups=0, starts=0, shared=0, attention=dict(wsb=1 << 16)), BUFFER)])
def test_shared_refusals(change, status):
    assert shared(describe(), **change) == status
    assert "bgg_shared_attention" in bgg.bgg_last_error()


def test_shared_null_empty_batch_and_workspace():
    d = describe()
    assert LIB.bgg_shared_attention(ctypes.byref(d), bgg._ATTENTION_ARGS.pack(*ATTENTION.values()), None, None) == NULL
    assert LIB.bgg_shared_attention(ctypes.byref(d), None, bgg._SHARED_ARGS.pack(*SHARED.values()), None) == NULL
    assert shared(d, attention=dict(batch=0), groups=0) == 0
    assert shared(d, attention=dict(batch=0), groups=1) == SHAPE
    size = bgg.bgg_shared_attention_workspace_size
    assert size(d, 4, 1) > bgg.bgg_attention_workspace_size(d, 4, 1)
    assert size(d, 4, 64) >= size(d, 4, 1)
    assert size(d, 3, 1) == size(d, 0, 1) == size(d, 4, 0) == size(d, 4, 4097) == 0
