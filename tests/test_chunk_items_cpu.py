"""How chunk attention's items are shared out, on the host: what its kernels' warps each
work out for themselves has to be alike, for nobody tells them."""

import importlib
import subprocess

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "chunk.cuh"
using namespace specv_chunk;

#define CHECK(x) \
  if (!(x)) { \
    std::printf("%s: len %d n %d group %d window %d prefix %d tile %d of %d..%d\n", #x, r.len, r.n, P.group, \
                P.window, r.prefix, row_tile, t0, t1); \
    return 1; \
  }

int main() {
  long items = 0;
  for (int group : {1, 3, 8, 64})
    for (int n : {1, 2, 33, 100, 300})
      for (int len : {0, 1, 63, 127, 128, 500})
        for (int window : {INT_MAX, 1, 70, 200})
          for (int prefix : {0, 1, 64, 130, 400}) {
            Params P = {};
            P.group = group;
            P.window = window;
            const Request r{0, n, len, prefix < len + n ? prefix : len + n, 0};
            for (int row_tile = 0; row_tile * kRowTile < n * group; row_tile++) {
              const Span span = span_of(P, r, row_tile);
              const bool pair = span.rows > kRows;
              for (int t0 = 0; t0 < span.tiles; t0++)
                for (int t1 = t0 + 1; t1 <= span.tiles; t1++) {
                  const Item w{0, 0, row_tile, t0, t1, span.gap, span.skip, span.rows, 0, n, len, r.prefix,
                               span.pos0, span.pos1, lowest(P, span.pos0), lowest(P, span.pos1), 1, 1, 0, 0, {}};
                  const Keys keys(w);
                  const Halves halves(keys, t0);
                  // the halves in the order of the tiles, each tile's upper one first, no other
                  int at = 0;
                  for (int i = 0; i < keys.tiles; i++)
                    for (int half = 1; half >= 0; half--) {
                      const int key = keys.first(i) + half * kHalf;
                      bool some = false;
                      for (int s = key; s < key + kHalf; s++)
                        some |= s < r.prefix || (s >= w.low0 && s <= w.pos1);
                      if (some) {
                        CHECK(at < halves.total && halves.key(at) == key);
                        at++;
                      }
                    }
                  CHECK(at == halves.total && at > 0);
                  // what each stream takes as its softmax and its MMAs go through them
                  for (int st = 0; st < 2; st++) {
                    int softmax = 0, mma = 0;
                    for (int i = pair ? 0 : st; i < halves.total; i += pair ? 1 : 2) softmax++;
                    for (int i = 0; i < halves.total; i++)
                      if (pair || (i & 1) == st) mma++;
                    CHECK(softmax == mma && softmax == halves.taken(pair, st));
                    for (int rows = 0; rows < 2; rows++) {
                      // nothing is read of an item that is flagged or behind a wait that gave up
                      CHECK(!halves.summed(pair, rows, st, true));
                      CHECK(halves.summed(pair, rows, st, false) == ((!pair || rows == st) && softmax > 0));
                    }
                  }
                  items++;
                }
            }
          }
  std::printf("%ld\n", items);
}
"""


def run(source, where):
    how = importlib.import_module("speculative_decoding_verify_sample_gb300.build")
    path = where / "items.cu"
    path.write_text(source)
    subprocess.run([how.nvcc_path(), *how.ARCH_FLAGS, "-O1", "-std=c++17", "-I", how.INCLUDE, "-I",
                    f"{how.PKG_DIR}/csrc", "-cudart", "shared", "-o", str(where / "items"), str(path)], check=True)
    done = subprocess.run([str(where / "items")], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
    return done.stdout


def test_streams_take_what_all_warps_work_out(tmp_path):
    """The halves of an item's keys, who takes them, and whose sums the rows at an item's end are made of."""
    assert int(run(PROGRAM, tmp_path)) > 10000


