"""The host code of the cache calls (bgg_cache.cpp: descriptors, frequency
tables, argument checks) under AddressSanitizer and
UndefinedBehaviorSanitizer: a small program over the extremes of every field.
Any report fails the test."""
import os
import subprocess
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_gemv_gemm_amd", "csrc")

MAIN = textwrap.dedent(r'''
    #include <climits>
    #include <cmath>
    #include <cstdio>
    #include <cstring>
    #include <vector>
    #include "bgg_cache.h"
    using namespace bgg;
    int main() {
      const int64_t ends[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 17, 64, 96, 255, 256, 65536, 65537, INT32_MAX,
                              (int64_t)INT32_MAX + 1, (int64_t)1 << 40, INT64_MAX};
      int described = 0, refused = 0;
      bgg_cache_desc d;
      for (int32_t type : {INT_MIN, 0, 1, 2, 3, 4, INT_MAX})
        for (int64_t pages : ends)
          for (int64_t size : ends)
            for (int64_t heads : ends)
              for (int64_t dim : ends)
                (bgg_cache_describe(type, pages, size, heads, dim, &d) == BGG_OK ? described : refused)++;
      if (bgg_cache_describe(BGG_TYPE_F16, 10, 16, 2, 64, &d) != BGG_OK) return 2;
      // the rotary and attention checks, one field at a time
      bgg_rotary_args r;
      bgg_attention_args a;
      void* p = (void*)(uintptr_t)(1 << 20);
      std::memset(&r, 0, sizeof r);
      r.type = 1, r.rotary_dim = 64, r.tokens = 3, r.q_heads = 4;
      r.q_dev = r.q_out_dev = p, r.k_dev = r.v_dev = p, r.k_cache_dev = r.v_cache_dev = p;
      r.q_stride = r.q_out_stride = 256, r.k_stride = r.v_stride = 128, r.magnitude = 1;
      r.positions_dev = (const int32_t*)p, r.slots_dev = (const int64_t*)p, r.freqs_dev = (const float*)p;
      if (check_rotary(&d, &r) != BGG_OK) return 3;
      int64_t* fields[] = {&r.rotary_dim, &r.tokens, &r.q_heads, &r.q_stride, &r.q_out_stride, &r.k_stride, &r.v_stride};
      for (int64_t* f : fields)
        for (int64_t v : ends) {
          const int64_t was = *f;
          *f = v;
          check_rotary(&d, &r);
          *f = was;
        }
      std::memset(&a, 0, sizeof a);
      a.type = 1, a.scale = 1, a.batch = 2, a.q_heads = 4, a.q_dev = p, a.out_dev = p, a.q_stride = a.out_stride = 256;
      a.k_cache_dev = a.v_cache_dev = p, a.page_table_dev = a.lengths_dev = (const int32_t*)p;
      a.table_width = a.table_stride = 4, a.workspace = p, a.workspace_bytes = 1 << 20;
      if (check_attention(&d, &a) != BGG_OK) return 4;
      int64_t* more[] = {&a.batch, &a.q_heads, &a.window, &a.q_stride, &a.out_stride, &a.table_width, &a.table_stride};
      for (int64_t* f : more)
        for (int64_t v : ends) {
          const int64_t was = *f;
          *f = v;
          check_attention(&d, &a);
          *f = was;
        }
      for (float s : {INFINITY, -INFINITY, NAN}) {
        a.scale = s;
        if (check_attention(&d, &a) == BGG_OK) return 5;
      }
      // frequency tables: exactly rotary_dim / 2 floats are written
      for (int64_t dim : {-2, 0, 1, 2, 4, 128, 256, 258})
        for (int scaling = -1; scaling < 5; ++scaling)
          for (double base : {1.0, 1.5, 1e4, 1e300, (double)INFINITY, (double)NAN})
            for (double factor : {0.5, 1.0, 64.0, 1e300, (double)NAN}) {
              std::vector<float> f(dim > 0 ? dim / 2 : 0);
              float m;
              float none;
              bgg_rotary_frequencies(dim, base, scaling, factor, 4096.0, 1.0, 32.0, f.empty() ? &none : f.data(), &m);
            }
      std::printf("%d %d\n", described, refused);
      return described > 0 && refused > 0 ? 0 : 6;
    }
''')


def _installed(name):
    out = subprocess.run(["gcc", f"-print-file-name={name}"], capture_output=True, text=True).stdout.strip()
    return os.path.isabs(out) and os.path.exists(out)


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
