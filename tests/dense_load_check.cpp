// Runs the dense operators' loads (dense_load.h) on the host, all threads of a
// workgroup one after the other, over matrices that lie against unmapped pages:
// a load that leaves the matrix's memory ends the program, which then names the
// case.  What was loaded is compared element by element.
#include <signal.h>
#include <sys/mman.h>
#include <unistd.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#define __device__
#define __forceinline__ inline
struct uint4 { unsigned x, y, z, w; };
static inline uint4 make_uint4(unsigned x, unsigned y, unsigned z, unsigned w) { return {x, y, z, w}; }
static struct { unsigned x; } threadIdx;

#include "dense_load.h"

using namespace oidn;

static char at[200];
static void outside(int) {
  (void)!write(1, "outside the matrix: ", 20);
  (void)!write(1, at, strlen(at));
  _exit(1);
}

static char *page, *end;        // what is mapped

// Element e of a matrix; pads hold 0xffff... .
template <int SIZE> static uint32_t value(long e) { return SIZE == 4 ? 0x10000001u + (uint32_t)e : (uint16_t)(1 + e % 60000); }

template <int SIZE>
static void set(char* p, uint32_t v) { memcpy(p, &v, SIZE); }
template <int SIZE>
static uint32_t get(const char* p) { uint32_t v = 0; memcpy(&v, p, SIZE); return v; }

// `rows` output rows, `len` summed elements at pitch ld, tiles from output row i0.
// gated: as many rows again, which the tile's second half reads.
template <int SIZE, int T, int D, bool STRIDED>
static int tiles(long rows, long len, long ld, long i0, bool at_end, bool gated = false) {
  typedef Loader<SIZE, T, D, STRIDED> L;
  const long half = gated ? rows : 0, outer = STRIDED ? len : rows + half, inner = STRIDED ? rows : len;
  const long elements = (outer - 1) * ld + inner;
  char* const base = at_end ? end - elements * SIZE : page;
  snprintf(at, sizeof at, "%d bytes, tile %d x %d, %s, %ld rows, length %ld, pitch %ld, from row %ld, %s\n", SIZE, T, D,
           STRIDED ? "strided" : gated ? "gated" : "l-fastest", rows, len, ld, i0, at_end ? "end" : "start");
  for (long e = 0; e < elements; ++e) set<SIZE>(base + e * SIZE, e % ld < inner ? value<SIZE>(e) : ~0u);
  for (threadIdx.x = 0; threadIdx.x < 256; ++threadIdx.x) {
    L loader(base, ld, i0, rows, 0, len, half);
    for (long l0 = 0; l0 < len; l0 += D) {
      uint4 u[L::kUnits];
      loader.load(u, l0);
      for (int k = 0; k < L::kUnits; ++k) {
        int r, s;
        L::place(k, r, s);
        for (int m = 0; m < L::kPer; ++m) {
          long i = i0 + (STRIDED ? L::kPer * s + m : gated ? r % (T / 2) : r);
          const long l = l0 + (STRIDED ? r : L::kPer * s + m);
          if (!STRIDED && i >= rows) i = rows - 1;
          if (gated && r >= T / 2) i += half;
          const uint32_t want = i < rows + half && l < len ? value<SIZE>(STRIDED ? l * ld + i : i * ld + l) : 0;
          const uint32_t got = get<SIZE>(reinterpret_cast<char*>(&u[k]) + SIZE * m);
          if (got != want) {
            printf("element (%ld, %ld) is %x, not %x: %s", i, l, got, want, at);
            return 1;
          }
        }
      }
    }
  }
  return 0;
}

template <int SIZE, int T, int D, bool STRIDED>
static int sweep() {
  // short rows at every pitch up to two loads, and lengths of every remainder
  for (long rows = 1; rows <= 10; ++rows)
    for (long len = 1; len <= (STRIDED ? 2 * D + 20 : 20); ++len)
      for (long ld = STRIDED ? rows : len; ld <= (STRIDED ? rows : len) + 16; ld += ld < 17 ? 1 : 7)
        for (int e = 0; e < 2; ++e)
          if (tiles<SIZE, T, D, STRIDED>(rows, len, ld, 0, e) || (!STRIDED && tiles<SIZE, T, D, STRIDED>(rows, len, ld, 0, e, true)))
            return 1;
  // rows that end inside a later tile
  for (long rows = T - 2; rows <= 2 * T + 10; rows += 3)
    for (long len : {1, 7, D - 1, D, D + 1, 2 * D + 3})
      for (long pad : {0, 1, 8})
        for (long i0 = 0; i0 < rows; i0 += T)
          if (tiles<SIZE, T, D, STRIDED>(rows, len, (STRIDED ? rows : len) + pad, i0, true)) return 1;
  return 0;
}

int main() {
  const long size = sysconf(_SC_PAGESIZE), bytes = 64 * size;
  char* const all = static_cast<char*>(mmap(nullptr, bytes + 2 * size, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
  if (all == MAP_FAILED || mprotect(all + size, bytes, PROT_READ | PROT_WRITE)) return 2;
  page = all + size;
  end = page + bytes;
  signal(SIGSEGV, outside);
  signal(SIGBUS, outside);
  if (sweep<2, 64, 64, true>() || sweep<2, 128, 64, true>() || sweep<4, 64, 32, true>() || sweep<2, 64, 64, false>() ||
      sweep<2, 128, 64, false>() || sweep<4, 64, 32, false>() || sweep<4, 32, 32, false>())
    return 1;
  printf("all inside\n");
  return 0;
}
