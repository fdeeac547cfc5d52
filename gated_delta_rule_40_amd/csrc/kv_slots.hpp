// kv_slots.hpp -- which slots of a page a call's new tokens take.  Plain
// constexpr arithmetic, the same in the kernels and on the host.
#pragma once

namespace gdr {

struct KvSlots {
  int u, w;   // slots [u, w) take new tokens; none if u >= w
  int had;    // slots [0, had) hold older tokens of the row
  int first;  // the new token of slot u
};

// Of page `page_no` (>= 0) of a row whose n (>= 0) new tokens lie at positions
// pos ... pos + n - 1.  pos may be any 32-bit value (negative positions are not
// written), so sums of it take 64 bits; what is returned lies within the page
// and the new tokens.
constexpr KvSlots kv_slots(int pos, int n, long long page_no, int page) {
  const long long at = pos, base = page_no * page;
  const long long lo = at > base ? at : base;  // base >= 0: negative positions end here
  const long long hi = at + n < base + page ? at + n : base + page;
  if (hi <= lo) return KvSlots{0, 0, 0, 0};
  return KvSlots{static_cast<int>(lo - base), static_cast<int>(hi - base),
                 at > base ? static_cast<int>(lo - base) : 0, static_cast<int>(lo - at)};
}

}  // namespace gdr
