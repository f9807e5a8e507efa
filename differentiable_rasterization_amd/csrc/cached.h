// cached.h — what the cache's kernels and attention over it share.
#pragma once

#include "tokens.h"

namespace gs {

// The caller's documents; without key ranges, keys are the tokens' rows.
inline Docs make_docs(const gs_documents& d, int64_t rows_q, int64_t rows_k) {
  Docs o = {};
  o.count = d.count;
  o.rows_q = (int)rows_q;
  o.rows_k = (int)rows_k;
  o.q_start = d.q_start;
  o.q_len = d.q_len;
  o.k_start = d.k_start ? d.k_start : d.q_start;
  o.k_len = d.k_len ? d.k_len : d.q_len;
  o.prefix = d.prefix;
  return o;
}

}  // namespace gs
