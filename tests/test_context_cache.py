"""Values kept per CUDA context (csrc/context_cache.h), with contexts played by numbers."""
import os
import re
import subprocess
import textwrap

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_schedule_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
#include "context_cache.h"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

static unsigned long long ctx = 0;
static int made = 0;
static unsigned long long id() { return ctx; }

int main() {
  using Cache = moe::ContextCache<int>;
  Cache c;
  int v = -1;
  auto make = [](int& n) { n = 10 * static_cast<int>(ctx) + ++made; return true; };
  // each context has its own value, made once
  ctx = 1; CHECK(c.get(id, make, v) && v == 11 && made == 1);
  CHECK(c.get(id, make, v) && v == 11 && made == 1);
  ctx = 2; CHECK(c.get(id, make, v) && v == 22 && made == 2);
  ctx = 1; CHECK(c.get(id, make, v) && v == 11 && made == 2);
  ctx = 2; CHECK(c.get(id, make, v) && v == 22 && made == 2);
  // a context made again after it was destroyed has another id
  ctx = 3; CHECK(c.get(id, make, v) && v == 33 && made == 3);
  // a failure is not kept
  Cache f;
  int tries = 0;
  ctx = 1;
  v = 5;
  CHECK(!f.get(id, [&](int&) { ++tries; return false; }, v) && v == 5 && tries == 1);
  CHECK(!f.get(id, [&](int&) { ++tries; return false; }, v) && tries == 2);
  CHECK(f.get(id, make, v) && made == 4 && f.get(id, make, v) && made == 4);
  // no context yet: the call that makes the value makes the context
  Cache z;
  ctx = 0;
  CHECK(z.get(id, [](int& n) { ctx = 7; n = 70; return true; }, v) && v == 70);
  CHECK(z.get(id, make, v) && v == 70 && made == 4);
  // the same from another thread, to which the context only then becomes current
  ctx = 0;
  CHECK(z.get(id, [](int& n) { ctx = 7; n = 71; return true; }, v) && v == 71);
  CHECK(z.get(id, make, v) && v == 70 && made == 4);
  // no context id at all: made at every call
  ctx = 0;
  const int before = made;
  CHECK(z.get(id, make, v) && z.get(id, make, v) && made == before + 2);
  // more contexts than slots: the oldest are made again
  Cache m;
  made = 0;
  for (ctx = 1; ctx <= Cache::kSlots + 1; ++ctx) CHECK(m.get(id, make, v));
  CHECK(made == Cache::kSlots + 1);
  ctx = Cache::kSlots + 1; CHECK(m.get(id, make, v) && made == Cache::kSlots + 1);
  ctx = 1; CHECK(m.get(id, make, v) && made == Cache::kSlots + 2);
  // threads that ask at the same time make it once
  Cache t;
  ctx = 9;
  made = 0;
  std::vector<std::thread> ts;
  for (int i = 0; i < 8; ++i) ts.emplace_back([&] { int n = 0; if (!t.get(id, make, n) || n != 91) std::exit(1); });
  for (auto& th : ts) th.join();
  CHECK(made == 1);
  std::printf("ok\n");
}
"""


def test_values_follow_the_context(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(textwrap.dedent(PROGRAM))
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_dense_and_4_bit_launches_keep_nothing_per_process():
    """What holds in one context only (a kernel's shared-memory limit, an occupancy) is
    never kept by a once_flag."""
    for f in ("dense_common.cuh", "ffn.cu", "fp4.cu", "fp4_gemm.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        assert not re.search(r"once_flag|call_once", text), f
        if f.endswith("_gemm.cu") or f == "ffn.cu":
            assert text.count("set_smem(") == text.count("cache.get(current_context_id") > 0, f
