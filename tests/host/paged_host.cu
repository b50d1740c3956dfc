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

// Rows of an output share an element: against marking every element.
void overlap() {
  int yes = 0, no = 0;
  for (int T = 1; T <= 6; ++T)
    for (int H = 1; H <= 6; ++H)
      for (int ts = 0; ts <= 40; ++ts)
        for (int hs = 0; hs <= 40; ++hs) {
          const int n = 4;
          bool used[6 * 40 * 2 + 8] = {}, meet = false;
          for (int t = 0; t < T; ++t)
            for (int h = 0; h < H; ++h)
              for (int c = 0; c < n; ++c) {
                bool& u = used[t * ts + h * hs + c];
                meet |= u, u = true;
              }
          ++(meet ? yes : no);
          EXPECT(kvq::rows_overlap(T, H, ts, hs, n) == meet, "%d x %d rows, strides %d and %d: %d", T, H, ts, hs, meet);
        }
  EXPECT(yes > 1000 && no > 1000, "%d and %d layouts", yes, no);
  const int64_t far = INT64_MAX - 7;
  EXPECT(!kvq::rows_overlap(INT32_MAX, INT32_MAX, far, 128, 128), "far tokens");
  EXPECT(!kvq::rows_overlap(2, 2, far, far - 128, 128), "far tokens and heads");
  EXPECT(kvq::rows_overlap(3, 3, far, far, 128), "the same strides");
}

// A warp that fills a ring ahead of its work, with a copy that does not arrive in time: behind the drain
// nothing is in flight any more, whatever the number of pages and the copy.
template <int STAGES>
void ring() {
  for (int pages = 1; pages <= 20; ++pages)
    for (int late = 0; late < pages; ++late) {
      int done[STAGES] = {}, pending[STAGES] = {};   // phases completed, copies in flight
      int issued = 0;
      // a barrier's wait for a parity returns once the phase of that parity is behind it
      auto ready = [&](int stage, uint32_t parity) { return (uint32_t)(done[stage] & 1) != parity; };
      auto land = [&](int stage) { ++done[stage], --pending[stage]; };
      auto issue = [&] { EXPECT(++pending[kvq::ring_stage<STAGES>(issued++)] == 1, "%d pages: a stage is filled twice", pages); };
      while (issued < pages && issued < STAGES) issue();
      bool failed = false;
      for (int it = 0; it < pages; ++it) {
        const int s = kvq::ring_stage<STAGES>(it);
        if (!failed) {
          EXPECT(!ready(s, kvq::ring_parity<STAGES>(it)), "%d pages: page %d seen before its copy", pages, it);
          if (it != late) {
            land(s);
            EXPECT(ready(s, kvq::ring_parity<STAGES>(it)), "%d pages: page %d not seen", pages, it);
          } else {
            failed = true;
            kvq::ring_drain<STAGES>(issued, [&](int stage, uint32_t parity) {
              if (!ready(stage, parity)) land(stage);
              EXPECT(ready(stage, parity), "%d pages, %d late: a wait for another phase", pages, late);
            });
            for (int k = 0; k < STAGES; ++k) EXPECT(pending[k] == 0, "%d pages, %d late: stage %d in flight", pages, late, k);
          }
        }
        if (!failed && issued < pages) issue();
      }
    }
}

}  // namespace

int main(int argc, char** argv) {
  const char* what = argc > 1 ? argv[1] : "";
  if (!std::strcmp(what, "rows")) rows();
  else if (!std::strcmp(what, "overlap")) overlap();
  else if (!std::strcmp(what, "ring")) ring<1>(), ring<2>(), ring<3>(), ring<4>();
  else EXPECT(false, "no check named '%s'", what);
  if (!wrong) std::puts("ok");
  return wrong != 0;
}
