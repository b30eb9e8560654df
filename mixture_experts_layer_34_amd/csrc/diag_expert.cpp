// Host views of what the expert operators' launches decide
// (include/mok_diag.h; test support).
#include "../../include/mok_diag.h"
#include "int4_matvec.h"

extern "C" int32_t mok_diag_expert_rows(int32_t begin, int32_t end, int32_t rows, int32_t* range) {
  if (!range) return 1;
  const mok::RowRange r = mok::cut_rows(begin, end, rows);
  range[0] = r.begin;
  range[1] = r.end;
  return 0;
}
