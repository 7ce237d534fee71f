"""The order of routed rows does not depend on which warp runs first.

place_range of csrc/route.cu is taken from its source and compiled for the host: a thread is a
fiber that runs from one __syncthreads to the next, and the warps of a CTA take their turns in a
chosen order.  Two accesses of one word without a barrier between them then come out wrong in one of
the orders, every time."""

import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import oracle
from mxfp8_block_scaled_02_gb300 import build

SHIM = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <algorithm>
#include <ucontext.h>
#include <vector>
using std::min;
#define __device__
#define __forceinline__ inline
constexpr int THREADS = 1024;
constexpr int GROUP = %(group)s;
struct Args { int64_t T; int E, k; const int* ids; int* rows; int* positions; };
struct Dim { int x; };
static Dim threadIdx;
static ucontext_t scheduler, fiber[THREADS];
static bool done[THREADS];
static int current;
static void __syncthreads() { swapcontext(&fiber[current], &scheduler); threadIdx.x = current; }
static int __popc(uint32_t v) { return __builtin_popcount(v); }
static uint32_t atomicOr(uint32_t* p, uint32_t v) { const uint32_t o = *p; *p |= v; return o; }

%(source)s

static Args args;
static std::vector<int> next_row;
static std::vector<uint32_t> mask;
static void body() {
  threadIdx.x = current;
  place_range(args, 0, args.T, next_row.data(), mask.data());
  done[current] = true;
}

// argv: T E k order; standard input: ids [T, k], first rows [E]; output: rows, positions
int main(int, char** argv) {
  args.T = atoi(argv[1]), args.E = atoi(argv[2]), args.k = atoi(argv[3]);
  const int order = atoi(argv[4]);
  std::vector<int> ids(args.T * args.k), rows(args.T * args.k, -1), positions(args.T * args.k, -2);
  next_row.resize(args.E);
  mask.assign(2 * args.E, 0xFFFFFFFFu);
  if (fread(ids.data(), 4, ids.size(), stdin) != ids.size()) return 1;
  if (fread(next_row.data(), 4, next_row.size(), stdin) != next_row.size()) return 1;
  args.ids = ids.data(), args.rows = rows.data(), args.positions = positions.data();
  std::vector<char> stacks(size_t(THREADS) * 16384);
  for (int t = 0; t < THREADS; ++t) {
    getcontext(&fiber[t]);
    fiber[t].uc_stack.ss_sp = &stacks[size_t(t) * 16384];
    fiber[t].uc_stack.ss_size = 16384;
    fiber[t].uc_link = &scheduler;
    makecontext(&fiber[t], body, 0);
  }
  uint32_t seed = 12345;
  for (bool left = true; left;) {
    left = false;
    int warps[THREADS / 32];
    for (int w = 0; w < THREADS / 32; ++w) warps[w] = order == 1 ? THREADS / 32 - 1 - w : w;
    if (order == 2)
      for (int w = THREADS / 32 - 1; w > 0; --w) {
        seed = seed * 1664525u + 1013904223u;
        std::swap(warps[w], warps[(seed >> 8) %% (w + 1)]);
      }
    for (int w : warps)
      for (int l = 0; l < 32; ++l) {
        current = 32 * w + l;
        if (done[current]) continue;
        swapcontext(&scheduler, &fiber[current]);
        left |= !done[current];
      }
  }
  fwrite(rows.data(), 4, rows.size(), stdout);
  fwrite(positions.data(), 4, positions.size(), stdout);
}
"""


def function(source: str, name: str) -> str:
    """The text of a function, up to the brace that closes it."""
    at = source.index("__device__ __forceinline__ void " + name + "(")
    depth, i = 0, source.index("{", at)
    while True:
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        i += 1
        if depth == 0:
            return source[at:i]


@pytest.fixture(scope="module")
def place(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    with open(os.path.join(build.CSRC, "route.cu")) as f:
        source = f.read()
    group = re.search(r"constexpr int GROUP = (\d+);", source).group(1)
    folder = tmp_path_factory.mktemp("place")
    (folder / "place.cpp").write_text(SHIM % {"group": group, "source": function(source, "place_range")})
    subprocess.run([gxx, "-std=c++17", "-O1", "-o", str(folder / "place"), str(folder / "place.cpp")], check=True)

    def run(ids: np.ndarray, first: np.ndarray, E: int, order: int):
        T, k = ids.shape
        r = subprocess.run([str(folder / "place"), str(T), str(E), str(k), str(order)],
                           input=ids.astype(np.int32).tobytes() + first.astype(np.int32).tobytes(), capture_output=True, check=True)
        out = np.frombuffer(r.stdout, dtype=np.int32)
        return out[:T * k], out[T * k:].reshape(T, k)

    return run


@pytest.mark.parametrize("order", ["first warp first", "last warp first", "drawn"])
@pytest.mark.parametrize("T,E,k", [(40, 64, 8), (64, 512, 4), (65, 16, 2), (128, 64, 8), (200, 33, 3), (300, 64, 8), (257, 512, 8)])
def test_rows_in_any_order_of_the_warps(place, T, E, k, order):
    """One to five groups of tokens by one CTA, the counts of which fill up to 32 warps."""
    rng = np.random.default_rng(T + E)
    z = rng.standard_normal((T, E)) * 3
    z[5] = -np.inf  # a token without experts
    want = oracle.route(z, k, "softmax", False)
    first = want["offsets"][:-1]
    rows, positions = place(want["ids"], first, E, ["first warp first", "last warp first", "drawn"].index(order))
    assert np.array_equal(positions, want["positions"])
    n = want["offsets"][-1]
    assert np.array_equal(rows[:n], want["rows"][:n]) and (rows[n:] == -1).all()
