"""Host side of the paged cache, the rotary positions and the attention:
descriptors, frequency tables, argument structs and refusals.  No GPU calls:
every refusal happens before anything is enqueued."""
import ctypes
import math
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


@pytest.mark.parametrize("type,elem", [("f16", 2), ("bf16", 2), ("e4m3", 1)])
@pytest.mark.parametrize("pages,page_size,heads,dim", [(1, 16, 1, 64), (7, 64, 8, 128), (1000, 65536, 4, 256),
                                                       (33, 32, 3, 96)])
def test_cache_sizes(type, elem, pages, page_size, heads, dim):
    d = describe(type, pages, page_size, heads, dim)
    assert d.page_bytes == page_size * heads * dim * elem
    assert d.total_bytes == pages * d.page_bytes
    assert (d.pages, d.page_size, d.kv_heads, d.head_dim, d.reserved) == (pages, page_size, heads, dim, 0)


@pytest.mark.parametrize("change,status", [
    (dict(type=0), FORMAT), (dict(type=4), FORMAT), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=1 << 17), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE),
    (dict(head_dim=80), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=512), SHAPE),
    (dict(pages=(1 << 31) - 1, page_size=65536, kv_heads=8), SHAPE)])
def test_cache_refusals(change, status):
    with pytest.raises(bgg.BggError) as e:
        describe(**change)
    assert e.value.status == status


def test_argument_structs_have_the_header_layout(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "bgg.h"\n#include <stdio.h>\n#define O(f) (int)offsetof(bgg_rotary_args, f)\n'
                   '#define A(f) (int)offsetof(bgg_attention_args, f)\n'
                   'int main(void){printf("%d %d %d %d %d %d %d %d %d\\n",(int)sizeof(bgg_cache_desc),'
                   '(int)sizeof(bgg_rotary_args),(int)sizeof(bgg_attention_args),O(q_dev),O(positions_dev),O(magnitude),'
                   'O(v_scale_dev),A(page_table_dev),A(workspace_bytes));return 0;}\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(bgg.bgg_cache_desc), bgg._ROTARY_ARGS.size, bgg._ATTENTION_ARGS.size, 32, 96, 120,
                   152, 104, 144]


# --- frequency tables -------------------------------------------------------
def test_frequencies_of_each_scaling():
    d, base, L = 128, 10000.0, 4096.0
    i = np.arange(0, d, 2, dtype=np.float64)
    f = base ** (-i / d)
    got, mag = bgg.bgg_rotary_frequencies(d, base)
    assert mag == 1.0 and np.array_equal(got, f.astype(np.float32))
    got, mag = bgg.bgg_rotary_frequencies(d, base, "linear", 8.0)
    assert mag == 1.0 and np.array_equal(got, (f / 8).astype(np.float32))
    got, mag = bgg.bgg_rotary_frequencies(d, base, "base", 8.0)
    want = (base * 8.0 ** (d / (d - 2))) ** (-i / d)
    # pow() of two libraries: a step of float32 apart at most
    assert mag == 1.0 and np.all(np.abs(got - want) <= 2.0 ** -23 * want)
    # the slowest pair of the stretched base turns factor times slower
    assert abs(got[-1] * 8.0 / f[-1] - 1) < 1e-6 and got[0] == 1.0
    got, mag = bgg.bgg_rotary_frequencies(d, base, "parts", 8.0, trained_length=L, low=1.0, high=32.0)
    turns = L * f / (2 * math.pi)
    g = np.clip((turns - 1) / 31, 0, 1)
    want = (1 - g) * f / 8 + g * f
    assert np.all(np.abs(got - want) <= 2.0 ** -23 * want)
    assert np.all(got[turns >= 32] == f[turns >= 32].astype(np.float32))
    assert np.all(got[turns <= 1] == (f[turns <= 1] / 8).astype(np.float32))
    assert mag == np.float32(1 + 0.1 * math.log(8))


@pytest.mark.parametrize("args,status", [
    ((0, 1e4), SHAPE), ((3, 1e4), SHAPE), ((258, 1e4), SHAPE), ((64, 1.0), SHAPE), ((64, math.inf), SHAPE),
    ((64, math.nan), SHAPE), ((64, 1e4, 4), FORMAT), ((64, 1e4, -1), FORMAT), ((64, 1e4, "linear", 0.5), SHAPE),
    ((64, 1e4, "linear", math.nan), SHAPE), ((2, 1e4, "base", 2.0), SHAPE), ((64, 1e4, "parts", 2.0, 0.0), SHAPE),
    ((64, 1e4, "parts", 2.0, 4096.0, 32.0, 32.0), SHAPE), ((64, 1e4, "parts", 2.0, math.inf), SHAPE)])
def test_frequency_refusals(args, status):
    with pytest.raises(bgg.BggError) as e:
        bgg.bgg_rotary_frequencies(*args)
    assert e.value.status == status


# --- refusals of the device calls -------------------------------------------
ROTARY = dict(type=1, layout=0, rotary_dim=64, tokens=3, q_heads=4, q=P, q_out=P, k=P, v=P, qs=256, qos=256, ks=128,
              vs=128, positions=P, slots=P, freqs=P, magnitude=1.0, reserved=0, kc=P, vc=P, ksc=0, vsc=0)
ATTENTION = dict(type=1, scale=0.1, batch=2, q_heads=4, window=0, q=P, out=P, qs=256, os=256, lse=P, kc=P, vc=P, ksc=0,
                 vsc=0, table=P, width=4, stride=4, lengths=P, ws=P, wsb=1 << 30)


def rotary(desc, **change):
    a = dict(ROTARY, **change)
    return LIB.bgg_rotary_append(ctypes.byref(desc) if desc is not None else None, bgg._ROTARY_ARGS.pack(*a.values()),
                                 None)


def attention(desc, **change):
    a = dict(ATTENTION, **change)
    return LIB.bgg_paged_attention(ctypes.byref(desc) if desc is not None else None,
                                   bgg._ATTENTION_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("change,status", [
    (dict(type=3), FORMAT), (dict(type=0), FORMAT), (dict(type=2), FORMAT), (dict(layout=2), FORMAT),
    (dict(ksc=P, vsc=P), FORMAT), (dict(reserved=1), SHAPE), (dict(rotary_dim=0), SHAPE), (dict(rotary_dim=63), SHAPE),
    (dict(rotary_dim=66), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 23) + 1), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(q_heads=4097, qs=1 << 20, qos=1 << 20), SHAPE), (dict(qs=248), SHAPE), (dict(qos=260), SHAPE),
    (dict(ks=120), SHAPE), (dict(vs=129), SHAPE), (dict(qos=264), SHAPE), (dict(q=0), NULL), (dict(q_out=0), NULL),
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(q=0, q_heads=0, k=0, v=0), NULL), (dict(positions=0), NULL),
    (dict(slots=0), NULL), (dict(freqs=0), NULL), (dict(kc=0), NULL), (dict(vc=0), NULL), (dict(q=P + 8), BUFFER),
    (dict(q_out=P + 2), BUFFER), (dict(k=P + 4), BUFFER), (dict(v=P + 8), BUFFER), (dict(positions=P + 2), BUFFER),
    (dict(slots=P + 4), BUFFER), (dict(freqs=P + 1), BUFFER), (dict(kc=P + 8), BUFFER), (dict(vc=P + 8), BUFFER)])
def test_rotary_refusals(change, status):
    assert rotary(describe(), **change) == status


def test_rotary_descriptor_and_no_tokens():
    assert rotary(None) == NULL
    d = describe()
    assert LIB.bgg_rotary_append(ctypes.byref(d), None, None) == NULL
    d.page_bytes += 1
    assert rotary(d) == DESC
    d = describe()
    d.magic ^= 1
    assert rotary(d) == DESC
    assert rotary(describe("e4m3")) == NULL  # scales are missing
    assert rotary(describe("e4m3"), ksc=P + 2, vsc=P) == BUFFER
    assert rotary(describe(), tokens=0) == 0
    # queries only: the cache's type does not matter, its buffers are not needed
    assert rotary(describe("bf16"), tokens=0, k=0, v=0, kc=0, vc=0, slots=0) == 0


@pytest.mark.parametrize("change,status", [
    (dict(type=3), FORMAT), (dict(type=2), FORMAT), (dict(ksc=P, vsc=P), FORMAT), (dict(scale=math.nan), SHAPE),
    (dict(scale=math.inf), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=4097), SHAPE), (dict(q_heads=3), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(q_heads=4098), SHAPE), (dict(window=-1), SHAPE), (dict(width=0), SHAPE),
    (dict(width=1 << 27, stride=1 << 27), SHAPE), (dict(stride=3), SHAPE), (dict(qs=255), SHAPE), (dict(os=128), SHAPE),
    (dict(q=0), NULL), (dict(out=0), NULL), (dict(kc=0), NULL), (dict(vc=0), NULL), (dict(table=0), NULL),
    (dict(lengths=0), NULL), (dict(ws=0), NULL), (dict(q=P + 8), BUFFER), (dict(out=P + 8), BUFFER),
    (dict(kc=P + 8), BUFFER), (dict(vc=P + 2), BUFFER), (dict(table=P + 2), BUFFER), (dict(lengths=P + 2), BUFFER),
    (dict(lse=P + 2), BUFFER), (dict(ws=P + 8), BUFFER), (dict(wsb=8), BUFFER)])
def test_attention_refusals(change, status):
    assert attention(describe(), **change) == status


def test_attention_descriptor_workspace_and_empty_batch():
    assert attention(None) == NULL
    d = describe()
    assert LIB.bgg_paged_attention(ctypes.byref(d), None, None) == NULL
    d.kv_heads = 1
    assert attention(d) == DESC
    assert attention(describe("e4m3")) == NULL
    assert attention(describe("e4m3"), ksc=P, vsc=P + 2) == BUFFER
    assert attention(describe(), batch=0) == 0
    d = describe()
    size = bgg.bgg_attention_workspace_size
    assert size(d, 4, 1) > 0 and size(d, 4, 64) >= size(d, 4, 1)
    assert size(d, 3, 1) == size(d, 0, 1) == size(d, 4, 0) == size(d, 4, 4097) == 0
    d.version += 1
    assert size(d, 4, 1) == 0
