"""The host checks of page assignment, rotary axes and shared prefix
attention under AddressSanitizer and UndefinedBehaviorSanitizer, over the
extremes of every field (as test_cache_sanitizers does for the other calls on
a cache).  Any report fails the test."""
import os
import subprocess
import textwrap

import pytest

from test_cache_sanitizers import CSRC, _installed

MAIN = textwrap.dedent(r'''
    #include <climits>
    #include <cstdio>
    #include <cstring>
    #include <vector>
    #include "bgg_cache.h"
    using namespace bgg;
    int main() {
      const int64_t ends[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 17, 64, 4095, 4096, 4097, 65536, 1 << 23, (1 << 23) + 1,
                              INT32_MAX, (int64_t)INT32_MAX + 1, (int64_t)1 << 40, INT64_MAX - 1, INT64_MAX};
      bgg_cache_desc d;
      if (bgg_cache_describe(BGG_TYPE_F16, 10, 16, 2, 64, &d) != BGG_OK) return 2;
      int passed = 0, refused = 0;
      auto over = [&](auto check, std::vector<int64_t*> fields) {
        for (int64_t* f : fields)
          for (int64_t* g : fields) {
            const int64_t f_was = *f, g_was = *g;
            for (int64_t v : ends)
              for (int64_t w : ends) {
                *f = v;
                *g = w;
                (check() == BGG_OK ? passed : refused)++;
              }
            *f = f_was;
            *g = g_was;
          }
      };
      auto at = [](int n) { return (void*)((uintptr_t)(n + 1) << 45); };  // buffers far apart

      bgg_assign_args a;
      std::memset(&a, 0, sizeof a);
      a.batch = 3, a.rows = 8, a.table_width = a.table_stride = 4, a.free_capacity = 10;
      a.lengths_dev = (const int32_t*)at(0), a.counts_dev = (const int32_t*)at(1), a.page_table_dev = (int32_t*)at(2);
      a.free_pages_dev = (int32_t*)at(3), a.free_count_dev = (const int32_t*)at(4), a.lengths_out_dev = (int32_t*)at(5);
      a.free_count_out_dev = (int32_t*)at(6), a.past_dev = (int32_t*)at(7), a.starts_dev = (int32_t*)at(8);
      a.positions_dev = (int32_t*)at(9), a.slots_dev = (int64_t*)at(10);
      if (check_assign(&d, &a) != BGG_OK) return 3;
      over([&] { return check_assign(&d, &a); }, {&a.batch, &a.rows, &a.table_width, &a.table_stride, &a.free_capacity});

      bgg_rotary_args r;
      bgg_rotary_axes_args x;
      std::memset(&r, 0, sizeof r);
      r.type = 1, r.rotary_dim = 64, r.tokens = 3, r.q_heads = 4, r.magnitude = 1;
      r.q_dev = at(0), r.q_out_dev = at(1), r.k_dev = at(2), r.v_dev = at(3), r.k_cache_dev = at(4), r.v_cache_dev = at(5);
      r.q_stride = r.q_out_stride = 256, r.k_stride = r.v_stride = 128;
      r.positions_dev = (const int32_t*)at(6), r.slots_dev = (const int64_t*)at(7), r.freqs_dev = (const float*)at(8);
      x.axes = 3, x.stride = 3, x.axis_of_pair_dev = (const uint8_t*)at(9);
      if (check_rotary_axes(&d, &r, &x) != BGG_OK) return 4;
      over([&] { return check_rotary_axes(&d, &r, &x); }, {&x.axes, &x.stride, &r.tokens, &r.rotary_dim, &r.q_heads, &r.q_stride});

      bgg_attention_args t;
      bgg_shared_args s;
      std::memset(&t, 0, sizeof t);
      t.type = 1, t.scale = 1, t.batch = 2, t.q_heads = 4, t.q_dev = at(0), t.out_dev = at(1), t.q_stride = t.out_stride = 256;
      t.k_cache_dev = at(2), t.v_cache_dev = at(3), t.page_table_dev = (const int32_t*)at(4), t.lengths_dev = (const int32_t*)at(5);
      t.table_width = t.table_stride = 4, t.workspace = at(6), t.workspace_bytes = (int64_t)1 << 40;
      s.groups = 1, s.group_starts_dev = (const int32_t*)at(7), s.shared_pages_dev = (const int32_t*)at(8);
      if (check_shared(&d, &t, &s) != BGG_OK) return 5;
      over([&] { return check_shared(&d, &t, &s); }, {&s.groups, &t.batch, &t.q_heads, &t.window, &t.table_width, &t.table_stride, &t.q_stride});

      // sections that add up to every sum a head can have, past it, and past 64 bits
      for (int64_t v : ends)
        for (int64_t w : ends)
          for (int32_t how : {INT_MIN, -1, 0, 1, 2, INT_MAX})
            for (int64_t n : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)2, (int64_t)4, (int64_t)5, INT64_MAX}) {
              const int64_t sections[4] = {v, w, 1, 1};
              std::vector<uint8_t> out(128);
              (bgg_rotary_axes(sections, n, how, out.data()) == BGG_OK ? passed : refused)++;
            }
      std::printf("%d %d\n", passed, refused);
      return passed > 0 && refused > 0 ? 0 : 6;
    }
''')


def test_host_checks_under_sanitizers(tmp_path):
    if not _installed("libasan.so") or not _installed("libubsan.so"):
        pytest.skip("gcc sanitizer runtimes not installed")
    main = tmp_path / "main.cpp"
    main.write_text(MAIN)
    exe = tmp_path / "checks"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                    "-I", CSRC, str(main), os.path.join(CSRC, "bgg_cache.cpp"), os.path.join(CSRC, "bgg_host.cpp"),
                    "-o", str(exe), "-lpthread"], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "ERROR" not in r.stderr and "runtime error" not in r.stderr, (r.returncode, r.stderr[-2000:])
