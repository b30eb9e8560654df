// Host views of what the expert operators' launches decide
// (include/mok_diag.h; test support).
#include "../../include/mok_diag.h"
#include "int4_rules.h"

namespace {

struct Report {
  int32_t* out;
  template <int NM, int NG, int RT, int GS, int KS, int NW, int SCH, bool WHOLE>
  hipError_t run(const mok::Int4Args&) const {
    const int32_t c[8] = {NM, NG, RT, GS, KS, NW, SCH, WHOLE};
    for (int i = 0; i < 8; ++i) out[i] = c[i];
    return hipSuccess;
  }
};

}  // namespace

extern "C" int32_t mok_diag_int4_config(int32_t rows, int32_t E, int32_t E_loc, int32_t routed, int32_t N, int32_t K,
                                        int32_t group, int32_t pair, int32_t* config) {
  if (!config || E < 1) return 1;
  static const int32_t some[2] = {};
  mok::Int4Args a{};
  a.offsets = routed ? some : nullptr;  // only whether there are any is asked
  a.rows = rows;
  a.E = E;
  a.E_loc = E_loc;
  a.N = N;
  a.K = K;
  a.group = group;
  a.pair = pair;
  return mok::launch_int4(a, Report{config}) == hipSuccess ? 0 : 1;
}

extern "C" int32_t mok_diag_expert_rows(int32_t begin, int32_t end, int32_t rows, int32_t* range) {
  if (!range) return 1;
  const mok::RowRange r = mok::cut_rows(begin, end, rows);
  range[0] = r.begin;
  range[1] = r.end;
  return 0;
}
