// Host-side: whether strided pieces of memory meet.
#pragma once
#include <algorithm>
#include <cstdint>

namespace dspark {

// Pieces of `bytes` bytes at base + the sum of i_k * stride[k], 0 <= i_k <
// size[k]; strides ascend, larger than what lies below them covers (pieces that
// touch are one).
struct Region {
  int64_t base, bytes, span, step;  // span: from the first byte to the last; step: the strides' greatest common divisor (0: none)
  int64_t size[4], stride[4];
  int dims, state;
  bool written;
};

inline int64_t common_divisor(int64_t a, int64_t b) {
  while (b) {
    const int64_t r = a % b;
    a = b;
    b = r;
  }
  return a;
}
// whether a multiple of g (0: only 0) lies in [lo, hi]
inline bool holds_multiple(int64_t lo, int64_t hi, int64_t g) {
  if (lo <= 0 && hi >= 0) return true;
  if (g == 0) return false;
  return hi < 0 ? -lo / g * g >= -hi : hi / g * g >= lo;
}

inline Region region_of(const void* base, const int64_t (&size)[4], const int64_t (&stride)[4], int64_t bytes, int state, bool written) {
  Region r{};
  r.base = reinterpret_cast<int64_t>(base);
  r.bytes = bytes;
  r.state = state;
  r.written = written;
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + 4, [&](int a, int b) { return stride[a] < stride[b]; });
  for (int i : order) {
    if (size[i] <= 1) continue;
    if (r.dims == 0 && stride[i] <= r.bytes) {
      r.bytes += stride[i] * (size[i] - 1);
      continue;
    }
    r.size[r.dims] = size[i];
    r.stride[r.dims++] = stride[i];
    r.step = common_divisor(r.step, stride[i]);
  }
  r.span = r.bytes;
  for (int k = 0; k < r.dims; ++k) r.span += r.stride[k] * (r.size[k] - 1);
  return r;
}

// one piece of memory (NULL: none)
inline Region piece_of(const void* base, int64_t bytes, int state, bool written) {
  constexpr int64_t one[4] = {1, 1, 1, 1}, none[4] = {0, 0, 0, 0};
  return region_of(base, one, none, base ? bytes : 0, state, written);
}

// Whether two regions share a byte: whether whole numbers c_k in [lo_k, hi_k]
// (differences of the two sides' indices along a stride) have a sum of c_k *
// stride_k between first and last, the distances of the bases at which pieces
// meet.  By the largest stride first; what is left has to be in reach of the
// smaller ones and near a multiple of their common divisor, so that nested
// strides leave two numbers or fewer for each.  Layouts that would take more
// than kLooks looks count as meeting.
struct RegionSearch {
  static constexpr int kLooks = 4096;
  int64_t stride[8], lo[8], hi[8], least[9], most[9], step[9];
  int n = 0, looks = 0;
  void add(int64_t s, int64_t from, int64_t to) {
    int k = 0;
    while (k < n && stride[k] > s) ++k;
    if (k == n || stride[k] != s) {
      for (int i = n++; i > k; --i) {
        stride[i] = stride[i - 1];
        lo[i] = lo[i - 1];
        hi[i] = hi[i - 1];
      }
      stride[k] = s;
      lo[k] = hi[k] = 0;
    }
    lo[k] += from;
    hi[k] += to;
  }
  bool find(int k, int64_t first, int64_t last) {
    if (++looks > kLooks) return true;
    first = std::max(first, least[k]);
    last = std::min(last, most[k]);
    if (first > last || !holds_multiple(first, last, step[k])) return false;
    if (k == n) return true;
    // c * stride + what the smaller ones can give reaches [first, last]
    const int64_t s = stride[k], a = first - most[k + 1], b = last - least[k + 1];
    int64_t c = a >= 0 ? (a + s - 1) / s : -(-a / s);
    const int64_t end = std::min(hi[k], b >= 0 ? b / s : -((-b + s - 1) / s));
    for (c = std::max(c, lo[k]); c <= end; ++c)
      if (find(k + 1, first - c * s, last - c * s)) return true;
    return false;
  }
};
inline bool regions_meet(const Region& x, const Region& y) {
  const int64_t apart = y.base - x.base, first = apart - (x.bytes - 1), last = apart + (y.bytes - 1);
  if (apart >= x.span || -apart >= y.span) return false;
  if (!holds_multiple(first, last, x.step == y.step ? x.step : common_divisor(x.step, y.step))) return false;
  RegionSearch q;
  for (int k = 0; k < x.dims; ++k) q.add(x.stride[k], 0, x.size[k] - 1);
  for (int k = 0; k < y.dims; ++k) q.add(y.stride[k], -(y.size[k] - 1), 0);
  q.least[q.n] = q.most[q.n] = q.step[q.n] = 0;
  for (int k = q.n - 1; k >= 0; --k) {
    q.least[k] = q.least[k + 1] + q.lo[k] * q.stride[k];
    q.most[k] = q.most[k + 1] + q.hi[k] * q.stride[k];
    q.step[k] = common_divisor(q.step[k + 1], q.stride[k]);
  }
  return q.find(0, first, last);
}

// Whether any two regions meet of which one is written, but for the two of one
// state (orders them by their bases).
inline bool any_meet(Region* r, int n) {
  std::sort(r, r + n, [](const Region& a, const Region& b) { return a.base < b.base; });
  for (int i = 0; i < n; ++i) {
    for (int j = i + 1; j < n && r[j].base < r[i].base + r[i].span; ++j)
      if ((r[i].written || r[j].written) && r[i].state != r[j].state && regions_meet(r[i], r[j])) return true;
  }
  return false;
}

}  // namespace dspark
