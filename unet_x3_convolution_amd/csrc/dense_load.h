// Loads of the dense operators' operands through registers, 16 bytes a thread,
// inside the matrix's memory at any size, pitch and element alignment.  Plain
// C++ over threadIdx and uint4, so that a test runs it on the host between
// unmapped pages.
#pragma once

namespace oidn {
namespace {

__device__ __forceinline__ uint4 load16_any(const char* p) {
  uint4 u;
  __builtin_memcpy(&u, p, 16);     // one 16-byte load: unaligned access is enabled on this target
  return u;
}
// A matrix's memory, for 16-byte loads near its end: a load that would pass the
// end is moved back inside and what it read is shifted, without a branch, so
// that all loads of a tile are in flight together.  A matrix of fewer than 16
// bytes is read once, element by element, into `all`.
template <int SIZE>
struct Extent {
  static constexpr int kPer = 16 / SIZE;
  const char* first;
  const char* last;        // where the last 16 bytes begin; before `first` if there are fewer
  uint4 all;
  __device__ __forceinline__ Extent(const void* base, long rows, long ld, long cols)
      : first(static_cast<const char*>(base)), last(first + ((rows - 1) * ld + cols) * SIZE - 16),
        all(make_uint4(0u, 0u, 0u, 0u)) {
    if (last >= first) return;
    const long n = (rows - 1) * ld + cols;
    unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < kPer - 1; ++k)
      if (k < n) {
        if constexpr (SIZE == 4) w[k] = reinterpret_cast<const unsigned*>(first)[k];
        else w[k / 2] |= (unsigned)reinterpret_cast<const unsigned short*>(first)[k] << (16 * (k % 2));
      }
    all = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Where to load for the unit at p of which n elements exist (n <= 0: none).
  __device__ __forceinline__ const char* from(const char* p, long n) const {
    const char* f = n > 0 ? p : first;
    f = f < last ? f : last;
    return f > first ? f : first;
  }
  // The unit's n elements, zeros after, from what was loaded at from(p, n).
  __device__ __forceinline__ uint4 shifted(uint4 u, const char* p, long n) const {
    const bool in = n > 0;
    const unsigned back = in ? (unsigned)(p - from(p, n)) * 8 : 0;    // bits, < 128
    const unsigned keep = n >= kPer ? 128u : in ? (unsigned)n * SIZE * 8 : 0u;
    unsigned long long lo = u.x | (unsigned long long)u.y << 32, hi = u.z | (unsigned long long)u.w << 32;
    if (back >= 64) lo = hi, hi = 0;
    const unsigned sh = back & 63;
    lo = lo >> sh | (sh ? hi << (64 - sh) : 0);
    hi >>= sh;
    lo = keep >= 64 ? lo : lo & ((1ull << keep) - 1);
    hi = keep >= 128 ? hi : keep > 64 ? hi & ((1ull << (keep - 64)) - 1) : 0;
    return make_uint4((unsigned)lo, (unsigned)(lo >> 32), (unsigned)hi, (unsigned)(hi >> 32));
  }
  // N units; at(k, p, n) gives the address of unit k and its elements.
  template <int N, class At>
  __device__ __forceinline__ void load(uint4 (&u)[N], At at) const {
    const char* p[N];
    long n[N];
#pragma unroll
    for (int k = 0; k < N; ++k) at(k, p[k], n[k]);
    uint4 raw[N];
    if (last < first) {
#pragma unroll
      for (int k = 0; k < N; ++k) raw[k] = all;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) raw[k] = load16_any(from(p[k], n[k]));
    }
#pragma unroll
    for (int k = 0; k < N; ++k) u[k] = shifted(raw[k], p[k], n[k]);
  }
};

// The loads of one operand's tiles through registers, in units of 16 bytes;
// SIZE: bytes of an element, T: output rows of a tile, D: its summed length.
// Unit k of a thread is unit `threadIdx.x + 256 k` of the tile: rows of D
// elements (l-fastest) or of T (STRIDED).
template <int SIZE, int T, int D, bool STRIDED>
struct Loader {
  static constexpr int kPer = 16 / SIZE;
  static constexpr int kUnits = T * D / kPer / 256;
  static constexpr int kPerRow = (STRIDED ? T : D) / kPer;
  const Extent<SIZE> all;
  const char* p[kUnits];     // of the next tile
  uint4 mask[STRIDED ? kUnits : 1];
  long step;                 // bytes to the next tile
  long i0, rows, ld, len, half;
  bool columns;              // STRIDED: every column of the tile exists

  // Row and unit in the row of unit k.
  static __device__ __forceinline__ void place(int k, int& r, int& s) {
    const int t = threadIdx.x + k * 256;
    r = t / kPerRow;
    s = t % kPerRow;
  }
  // Tiles start at output row i0_ (of rows_) and summed element l0 (of len_).
  // half_: tile rows from T / 2 on come from `half` further matrix rows
  // (l-fastest only; the up projection's rows of a gated product).
  __device__ __forceinline__ Loader(const void* base, long ld_, long i0_, long rows_, long l0, long len_, long half_)
      : all(base, STRIDED ? len_ : rows_ + half_, ld_, STRIDED ? rows_ : len_), step((STRIDED ? D * ld_ : D) * SIZE),
        i0(i0_), rows(rows_), ld(ld_), len(len_), half(half_), columns(i0_ + T <= rows_) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      long n;
      at(k, l0, p[k], n);
      if constexpr (STRIDED) {
        int r, s;
        place(k, r, s);
        n = rows - (i0 + kPer * s);
        // a unit past the columns reads its row's first ones, and keeps none
        if (n <= 0) p[k] = all.first + (l0 + r) * ld * SIZE;
        auto word = [&](int m) {         // bits of 32-bit word m whose elements exist
          const long left = n * SIZE - 4 * m;
          return left >= 4 ? ~0u : left == 2 ? 0xffffu : 0u;
        };
        mask[k] = make_uint4(word(0), word(1), word(2), word(3));
      }
    }
  }
  __device__ __forceinline__ void at(int k, long l0, const char*& q, long& n) const {
    int r, s;
    place(k, r, s);
    if constexpr (!STRIDED) {
      long i = i0 + (half ? r & (T / 2 - 1) : r);
      i = (i < rows ? i : rows - 1) + (half && r >= T / 2 ? half : 0);
      const long l = l0 + kPer * s;
      q = all.first + SIZE * (i * ld + l);
      n = len - l;
    } else {
      const long l = l0 + r, i = i0 + kPer * s;
      q = all.first + SIZE * (l * ld + i);
      n = l < len ? rows - i : 0;
    }
  }
  // The next tile, which starts at l0.
  __device__ __forceinline__ void load(uint4 (&u)[kUnits], long l0) {
    // a load that starts at a strided row's last column ends kPer - 1 elements
    // after it, in the rows that follow: one, or several where the pitch is less
    const bool inside = STRIDED && !columns ? (len - l0 - D) * ld >= kPer - 1 : l0 + D <= len;
    if (inside) {
#pragma unroll
      for (int k = 0; k < kUnits; ++k) u[k] = load16_any(p[k]);
      if (STRIDED && !columns) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
          const uint4 m = mask[STRIDED ? k : 0];
          u[k] = make_uint4(u[k].x & m.x, u[k].y & m.y, u[k].z & m.z, u[k].w & m.w);
        }
      }
    } else {
      all.load(u, [&](int k, const char*& q, long& n) { at(k, l0, q, n); });
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) p[k] += step;
  }
};

}  // namespace
}  // namespace oidn
