// views.cuh — host checks of strided tensor views (bsa_view_t), shared by the
// entry points that take them.
#pragma once
#include <stdint.h>

#include <cstdio>

#include "bsa.h"

// Defined in api.cu (internal, not part of the C ABI).
bsa_status bsa_internal_fail(bsa_status s, const char* msg);
bsa_status bsa_internal_plan_sizes(bsa_plan_t plan, const Geo** g, int* is_bf16, int* device);

namespace bsa {

// A checked view: strides in elements, 0 along axes of length 1.
struct View {
  char* p;
  long long b, n, h;
};

// Checks `v` as a [B, N, H, D] tensor of esz-byte elements (the rules of
// bsa_view_t) and copies it to *out.  `written` also asks that no two elements
// share memory.
inline bsa_status check_view(const bsa_view_t* v, const char* name, long long B, long long N, long long H,
                             long long D, int esz, bool written, View* out) {
  char msg[160];
  const char* why = nullptr;
  if (v == nullptr || v->ptr == nullptr) {
    why = "is NULL";
  } else if (reinterpret_cast<uintptr_t>(v->ptr) & 15u) {
    why = "must be 16-byte aligned";
  } else {
    long long st[3] = {B > 1 ? v->batch : 0, N > 1 ? v->token : 0, H > 1 ? v->head : 0};
    long long len[3] = {B, N, H};
    *out = View{static_cast<char*>(v->ptr), st[0], st[1], st[2]};
    for (int i = 0; i < 3; ++i) {
      if (st[i] < 0 || st[i] >= (1ll << 38) / esz) why = "has a stride that is negative or too large";
      else if ((st[i] * esz) & 15) why = "has a stride that is no multiple of 16 bytes";
    }
    if (why == nullptr && written) {
      // in the order of the strides, each axis has to step over all that the
      // shorter ones cover
      for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 3; ++j)
          if (st[j] < st[i]) {
            const long long s = st[i], l = len[i];
            st[i] = st[j]; len[i] = len[j];
            st[j] = s; len[j] = l;
          }
      long long covered = D;
      for (int i = 0; i < 3; ++i) {
        if (len[i] == 1) continue;
        if (st[i] < covered) why = "is written to and has elements that overlap";
        covered += st[i] * (len[i] - 1);
      }
    }
  }
  if (why == nullptr) return BSA_OK;
  snprintf(msg, sizeof(msg), "%s %s", name, why);
  return bsa_internal_fail(BSA_ERR_INVALID_ARG, msg);
}

inline bool same_view(const View& a, const View& b) {
  return a.p == b.p && a.b == b.b && a.n == b.n && a.h == b.h;
}

}  // namespace bsa
