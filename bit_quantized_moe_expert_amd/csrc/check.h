// Host-side checks and workspace carving shared by the C ABI files.
#pragma once
#include <initializer_list>

#include "internal.h"
#include "status.h"

namespace nf4moe {

inline bool dt_ok(int dt) { return dt == NF4MOE_DT_F32 || dt == NF4MOE_DT_BF16; }
inline size_t dt_bytes(int dt) { return dt == NF4MOE_DT_BF16 ? 2 : 4; }

// An array that a call writes or reads (absent: no address or no bytes).
struct Span {
  const char *name;
  const void *p;
  uint64_t n;
};
inline bool overlap(const Span &a, const Span &b) {
  const uint64_t p = (uint64_t)a.p, q = (uint64_t)b.p;
  return p && q && a.n && b.n && p < q + b.n && q < p + a.n;
}

// No output shares a byte with an input or with another output. An input that an output
// may be is left out of `ins` by the caller where it is that very array (see but()).
inline nf4moe_status_t check_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span *o = outs.begin(); o != outs.end(); ++o) {
    for (const Span *q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return fail(NF4MOE_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
    for (const Span &q : ins)
      if (overlap(*o, q)) return fail(NF4MOE_ERR_INVALID_ARG, "%s overlaps %s", o->name, q.name);
  }
  return NF4MOE_OK;
}
inline Span but(Span in, const void *out) { return {in.name, in.p == out ? nullptr : in.p, in.n}; }

// Bump allocator over the caller's workspace (sizes alone with a null base).
struct Bump {
  char *base;
  size_t off = 0;
  template <class T>
  T *take(size_t count) {
    T *p = base ? (T *)(base + off) : nullptr;
    off = align_up(off + count * sizeof(T));
    return p;
  }
};

}  // namespace nf4moe
