// Index arithmetic of the rotary and paged-cache kernels, enumerated on the host with the
// functions that the kernels call.  No CUDA call is made.
//   paged_host <check>: prints what is wrong and returns 1, or prints "ok"
#include <cstdio>
#include <cstring>

#include "kvq_rope.cuh"

namespace {

int wrong = 0;
#define EXPECT(ok, ...)                                             \
  do {                                                              \
    if (!(ok) && ++wrong <= 20) std::printf(__VA_ARGS__), std::puts(""); \
  } while (0)

// Every plan whose rows are exchanged through shared memory: partners lie within the warp's room, in
// the same row, and the lanes left over read their own elements.
void rows() {
  int plans = 0;
  for (int hd = 8; hd <= 256; hd += 8)
    for (int rd = 2; rd <= hd; rd += 2)
      for (int copy = 0; copy < 2; ++copy) {
        kvq_rope_plan plan = {};
        plan.head_dim = hd, plan.rotary_dim = rd;
        if (kvq::rope_pairs(plan) != 0 || (copy && rd == hd)) continue;
        ++plans;
        const int half = rd / 2, vecs = kvq::row_vectors(plan, copy), rows = 32 / vecs;
        EXPECT(vecs >= 1 && vecs <= 32, "head_dim %d, rotary_dim %d: %d vectors", hd, rd, vecs);
        for (int lane = 0; lane < 32; ++lane) {
          const int c0 = kvq::row_channel(lane, vecs), r = lane / vecs;
          for (int ch = c0; ch < c0 + 8; ++ch) {
            const int at = kvq::row_partner(lane, c0, ch, half);
            EXPECT(at >= 0 && at < 256, "head_dim %d, rotary_dim %d, copy %d: lane %d reads element %d", hd, rd, copy, lane, at);
            if (r >= rows) {
              EXPECT(at / 8 == lane, "head_dim %d, rotary_dim %d, copy %d: lane %d reads a row", hd, rd, copy, lane);
              continue;
            }
            EXPECT(c0 == 8 * (lane % vecs), "head_dim %d, rotary_dim %d: channel %d of lane %d", hd, rd, c0, lane);
            const int want = ch < half ? ch + half : ch < 2 * half ? ch - half : ch;
            EXPECT(at == 8 * vecs * r + want, "head_dim %d, rotary_dim %d: element %d of row %d", hd, rd, ch, r);
          }
        }
      }
  EXPECT(plans > 2000, "only %d plans", plans);
}

}  // namespace

int main(int argc, char** argv) {
  const char* what = argc > 1 ? argv[1] : "";
  if (!std::strcmp(what, "rows")) rows();
  else EXPECT(false, "no check named '%s'", what);
  if (!wrong) std::puts("ok");
  return wrong != 0;
}
