// The kernel instances that a dense feed-forward call launches, as text, from
// the plan the library itself uses.
#include <stdio.h>

#include "ffn_plan.h"

using namespace moe;

namespace {

struct Out {
  char* p;
  int left;
  template <class... A>
  void add(const char* fmt, A... a) {
    const int n = snprintf(p, left, fmt, a...);
    if (n > 0 && n < left) {
      p += n;
      left -= n;
    }
  }
  // sums: a row product, whose reduction may be split
  void tile(const char* name, const Plan& r, bool sums) {
    if (r.width == 256)
      add("%s 256x256x1;", name);
    else
      add("%s %dx%dx%d%s;", name, r.height, r.width, r.groups,
          !sums ? "" : r.splits > 1 ? " split" : " whole");
  }
  void thin(const char* name, const ThinPlan& r) {
    add("%s thin %d blocks %d rows%s;", name, r.blocks, r.rows,
        r.staged ? " staged" : "");
  }
};

}  // namespace

// want: the gradients asked for, 1 dx, 2 dw_gu, 4 dw2; 0: the forward.
extern "C" void ffn_forms(int64_t T, int64_t d, int64_t f, int want,
                          char* out, int bytes) {
  Out o{out, bytes};
  out[0] = 0;
  if (want == 0) {
    if (thin_form(T, d, f)) {
      o.thin("fc1", thin_plan(T, f));
      o.thin("y", thin_plan(T, d));
    } else {
      o.tile("fc1", fc1_plan(T, d, f), false);
      o.tile("y", row_plan(T, d, f), true);
    }
    return;
  }
  const bool dx = want & 1, dw_gu = want & 2, dw2 = want & 4;
  if (!dx && !dw_gu) {
    o.tile("dw", weight_plan(T, d, f), false);
    return;
  }
  if (dw2 && dact_pair(T, d, f).width) {
    o.tile("dact+dw2", dact_pair(T, d, f), false);
  } else {
    if (dw2) o.tile("dw", weight_plan(T, d, f), false);
    o.tile("dact", dact_plan(T, d, f), false);
  }
  if (dx && dw_gu && dx_pair(T, d, f).width) {
    o.tile("dx+dw_gu", dx_pair(T, d, f), true);
    return;
  }
  if (dw_gu) o.tile("dw", weight_plan(T, 2 * f, d), false);
  if (dx) o.tile("dx", row_plan(T, d, 2 * f), true);
}
