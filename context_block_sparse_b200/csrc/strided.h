// Checks of a call's arrays on the host: alignment, and whether two strided ones share memory.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <numeric>

namespace splitkv {

// Arrays of 32-bit words on their boundary (NULL passes).
template <typename... Ps>
inline bool all_aligned4(Ps... ps) {
  return ((reinterpret_cast<uintptr_t>(ps) % 4 == 0) && ...);
}

// Rows of `row` contiguous bytes at every sum of strides (bytes, >= 0) from ptr on.
struct Strided {
  const void* ptr;
  int64_t row;
  int n;
  int64_t size[4], stride[4];
};

// True where no byte of x is one of y's.  Either their extents do not meet, or the arrays are woven: modulo the common
// divisor g of some of their strides every element lies in a window of g (what the other dimensions span), and the two
// windows do not meet (heads of a fused projection, keys beside values in the pages of one cache).  False where
// neither shows it.
inline bool apart(const Strided& x, const Strided& y) {
  const auto extent = [](const Strided& a, int woven) {
    constexpr int64_t kAll = int64_t(1) << 61;   // past every address
    int64_t w = a.row;
    for (int i = 0; i < a.n; ++i) {
      if (woven >> i & 1 || a.size[i] < 2 || a.stride[i] == 0) continue;
      if (a.size[i] - 1 > (kAll - w) / a.stride[i]) return kAll;
      w += (a.size[i] - 1) * a.stride[i];
    }
    return w;
  };
  const int64_t x0 = int64_t(reinterpret_cast<uintptr_t>(x.ptr)), y0 = int64_t(reinterpret_cast<uintptr_t>(y.ptr));
  if (x0 + extent(x, 0) <= y0 || y0 + extent(y, 0) <= x0) return true;
  const auto woven = [&](int wx, int wy) {
    int64_t g = 0;
    for (int i = 0; i < x.n; ++i)
      if (wx >> i & 1 && x.size[i] > 1) g = std::gcd(g, x.stride[i]);
    for (int i = 0; i < y.n; ++i)
      if (wy >> i & 1 && y.size[i] > 1) g = std::gcd(g, y.stride[i]);
    if (g == 0) return false;
    const int64_t off = ((y0 - x0) % g + g) % g;
    return off >= extent(x, wx) && off + extent(y, wy) <= g;
  };
  // (the same dimensions of both first: what callers have)
  if (x.n == y.n)
    for (int w = 1; w < 1 << x.n; ++w)
      if (woven(w, w)) return true;
  for (int wx = 0; wx < 1 << x.n; ++wx)
    for (int wy = 0; wy < 1 << y.n; ++wy)
      if (woven(wx, wy)) return true;
  return false;
}

}  // namespace splitkv
