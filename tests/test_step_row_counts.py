"""Rows and blocks that are counted up to 2^31 - 1: the loops over them, as they stand in the sources, compiled for the host with
their types and run over the last turns of the largest counts (no GPU needed). A count in `int` that steps past 2^31 turns
negative there and goes on in front of the tensors."""
import os
import re
import subprocess

import pytest

import routed_expert_ffn_softmax_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return f.read()


def found(pattern, name):
    m = re.findall(pattern, source(name))
    assert len(m) == 1, (pattern, m)
    return m[0]


def run(tmp_path, body):
    src, exe = tmp_path / "loop.cpp", tmp_path / "loop"
    src.write_text("""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
struct { unsigned x; } blockIdx, gridDim;
struct { int N; } p;
static int64_t seen[8];
static int turns, ahead;
static bool bad(int64_t at, int64_t count) { return at < 0 || at >= count; }
""" + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("grid", [1, 7, 152, 304, 1216, 4864])
def test_norm_rows(tmp_path, grid):
    """The rows a block works on and those whose loads it starts ahead, from two turns before the last row on."""
    loop = found(r"(for \([^;{]*n = blockIdx\.x; n < [^{]*\)) \{", "add_rms_norm.cu")
    param, cond = found(r"auto load = \[&\]\((\w+ n)\) \{[^}]*if \(mine\[i\] && (n < [^{]*)\) \{", "add_rms_norm.cu")
    ahead = found(r"\n    (load\(n \+ [^;]*\);)", "add_rms_norm.cu")
    rows = " ".join(re.findall(r"const \w+ rows = [^;]*;", source("add_rms_norm.cu")))
    run(tmp_path, f"""
int main() {{
  gridDim.x = {grid};
  for (int N : {{2147483647, 2147483646, 2147483647 - {grid}}}) {{
    p.N = N;
    for (unsigned back = 0; back < 2 * gridDim.x; ++back) {{
      blockIdx.x = N - 1 - back;
      int turn = 0;
      {rows}
      turns = ahead = 0;
      auto load = [&]({param}) {{
        if ({cond}) {{ ++ahead; seen[6] = n; if (bad(seen[6], N)) ahead = 100; }}
      }};
      {loop} {{
        seen[turns] = n;
        if (bad(seen[turns], N) || ++turns > 3) {{ turns = 100; break; }}
        {ahead}
      }}
      (void)turn;
      const int want = 1 + static_cast<int>(back / gridDim.x);
      if (turns != want || ahead != want - 1) {{
        std::printf("N %d, row N - 1 - %u: %d turns, %d ahead, row %lld\\n", N, back, turns, ahead, (long long)seen[6]);
        return 1;
      }}
    }}
  }}
}}
""")


@pytest.mark.parametrize("grid", [1, 152, 912])
def test_blocks_read_back(tmp_path, grid):
    loop, item = found(r"(for \(\w+ (\w+) = blockIdx\.x \* kLoadWarps[^{]*\)) \{", "kv4_load.cu")
    total = found(r"const (\w+) total = ", "kv4_load.cu")
    warps = int(found(r"constexpr int kLoadThreads = (\d+);", "kv4_load.cu")) // 32
    run(tmp_path, f"""
constexpr int kLoadWarps = {warps};
int main() {{
  gridDim.x = {grid};
  for (int64_t count : {{2147483647, 2147483640, 2147483647 - {grid}}}) {{
    const {total} total = count;
    for (unsigned back = 0; back < 2 * gridDim.x * kLoadWarps; ++back) {{
      const int64_t at = count - 1 - back;
      blockIdx.x = static_cast<unsigned>(at / kLoadWarps);
      const int warp = static_cast<int>(at % kLoadWarps);
      turns = 0;
      {loop} {{
        seen[turns] = {item};
        if (bad(seen[turns], count) || ++turns > 3) {{ turns = 100; break; }}
      }}
      if (turns != 1 + static_cast<int>(back / (gridDim.x * kLoadWarps))) {{
        std::printf("%lld blocks, block %lld: %d turns\\n", (long long)count, (long long)at, turns);
        return 1;
      }}
    }}
  }}
}}
""")
