// How the attention over a paged cache is cut into work, shared by its kernels.
//
// An item is a run of new tokens of one sequence with `gt` query heads of a key/value head: the rows
// (token, head) of a tile.  Its cost is its key blocks and a constant, for an item of two tiles as for one of one: the
// block is fetched once for both, and a lone tile's two halves of a CTA take turns at its blocks.  (Two units a block
// for two tiles: 182 us for the ragged window of 8 sequences, 163 at best with a larger constant; one unit: 142.)  All items stand on a line, sequence by sequence, tile by tile, the heads of a tile side
// by side, and each CTA takes an equal stretch of it, cut between key blocks: ragged batches spread
// evenly, and a long context with few rows is shared by all SMs.  An item that lies in several
// stretches leaves its parts (o unnormalised, maximum, sum) in the workspace, at most two a CTA, and
// a last launch joins them in a fixed order.
#pragma once
#include "diff.h"
#include "paged.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxCtas = 304;

struct Cut {
  int gt;      // query heads handled together (divides the heads of a key/value head)
  int nv;      // groups of gt query heads
  int per_kv;  // ... of a key/value head
  int tile;    // tokens of a tile
  int step;    // tokens of an item (tile, or 2 tile: then an item of more than `tile` tokens fills two)
  int shift;   // a block holds 1 << shift keys
  int over;    // cost of an item beside its blocks, in blocks
  int least;   // blocks of a stretch, at the least
  int ctas;
};
struct Work {
  Seqs seqs;
  Cut cut;
  int causal, window;
};
struct Tail {  // the item that begins in a CTA's stretch and goes on behind it
  int b, tile, vh, parts;  // parts 0: none
};
// Workspace: Tail[ctas], then two slots per CTA of `rows` rows: o [rows][D], (max in powers of two, sum) [rows].  Slot 2p
// holds CTA p's part of an item that began before, slot 2p + 1 of one that begins here and goes on.
struct Space {
  Tail* tail;
  float* slots;
  int64_t slot;  // floats of a slot
  int rows, D;
  static int64_t header(int ctas) { return (ctas * static_cast<int64_t>(sizeof(Tail)) + 255) / 256 * 256; }
  static size_t bytes(int ctas, int rows, int D) {
    return static_cast<size_t>(header(ctas)) + 2ull * ctas * rows * (D + 2) * sizeof(float);
  }
  static Space at(void* ws, int ctas, int rows, int D) {
    Space s;
    s.tail = static_cast<Tail*>(ws);
    s.slots = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + header(ctas));
    s.slot = static_cast<int64_t>(rows) * (D + 2);
    s.rows = rows, s.D = D;
    return s;
  }
  __device__ __forceinline__ float* o(int k, int row) const { return slots + k * slot + static_cast<int64_t>(row) * D; }
  __device__ __forceinline__ float2* ml(int k, int row) const {
    return reinterpret_cast<float2*>(slots + k * slot + static_cast<int64_t>(rows) * D) + row;
  }
};

struct Blocks {
  int j0, n;  // key blocks j0 .. j0 + n - 1 (at least one, which may be hidden from every row)
};
// The key blocks that tokens t0 .. t1 - 1 of a sequence see.
__device__ __forceinline__ Blocks blocks_of(const Work& w, const Seq& s, int t0, int t1) {
  const int hi = w.causal ? min(max(s.start + t1, 0), s.len) : s.len;
  const int64_t l = static_cast<int64_t>(s.start) + t0 - w.window + 1;
  const int lo = w.window > 0 && l > 0 ? static_cast<int>(l) : 0;
  if (hi <= lo) return Blocks{0, 1};
  const int j0 = lo >> w.cut.shift;
  return Blocks{j0, ((hi - 1) >> w.cut.shift) + 1 - j0};
}

// The units of a tile of a sequence, all groups of heads.
__device__ __forceinline__ int64_t tile_units(const Work& w, const Seq& s, int tile) {
  const int t0 = tile * w.cut.step, t1 = min(s.n, t0 + w.cut.step);
  const Blocks k = blocks_of(w, s, t0, t1);
  return static_cast<int64_t>(k.n) + w.cut.over;
}
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The stretch of one CTA and the item in which it begins (b < 0: none), by one warp of its own (every lane gets
// them).  Each CTA plans for itself: a planning launch in front took 4 to 5 us of every call.  The sequences are looked at
// 32 at a time, twice: 21 us a thousand of them (0.24 ms for 10000, 21 ms for a million), and more where sequences have
// more than kFew tiles.  So it is done in front of the CTA's first barrier, where the other warps wait for as long
// as it takes, and not behind a bounded wait.
struct Plan {
  int64_t from, to, stretch;
  int64_t pos;  // of the item on the line
  int b, tile, vh;
};
__device__ __forceinline__ Plan plan(const Work& w, int p) {
  const int lane = threadIdx.x & 31, B = w.seqs.B, step = w.cut.step;
  constexpr int kFew = 4;  // tiles of a sequence that its lane looks at alone; the others are the warp's
  auto units = [&](int b0) {  // of sequence b0 + lane
    Seq s{};
    if (b0 + lane < B) s = seq_at(w.seqs, b0 + lane);
    int64_t v = 0;
    for (int t = 0; t < kFew && static_cast<int64_t>(t) * step < s.n; ++t) v += tile_units(w, s, t);
    for (unsigned many = __ballot_sync(0xffffffffu, s.n > static_cast<int64_t>(kFew) * step); many != 0; many &= many - 1) {
      const int from = __ffs(many) - 1;
      const Seq q = seq_at(w.seqs, b0 + from);
      int64_t u = 0;
      for (int64_t t = kFew + lane; t * step < q.n; t += 32) u += tile_units(w, q, static_cast<int>(t));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      if (lane == from) v += u;
    }
    return v * w.cut.nv;
  };
  int64_t total = 0;
  const int64_t mine = units(0);  // (the first 32 sequences are looked at once)
  for (int b0 = 0; b0 < B; b0 += 32) total += b0 == 0 ? mine : units(b0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int64_t even = (total + w.cut.ctas - 1) / w.cut.ctas;
  Plan r{};
  r.stretch = even > w.cut.least ? even : w.cut.least;
  r.from = r.stretch * p, r.to = min(r.from + r.stretch, total);
  r.b = -1;
  if (r.from >= total) return r;
  int64_t at = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {  // the first sequence that ends behind `from`
    const int64_t v = b0 == 0 ? mine : units(b0), cum = at + warp_scan(v, lane);
    const unsigned behind = __ballot_sync(0xffffffffu, cum > r.from);
    if (behind == 0) {
      at = __shfl_sync(0xffffffffu, cum, 31);
      continue;
    }
    const int from = __ffs(behind) - 1;
    at = __shfl_sync(0xffffffffu, cum - v, from);
    r.b = b0 + from;
    break;
  }
  const Seq s = seq_at(w.seqs, r.b);
  for (int64_t t0 = 0; t0 * step < s.n; t0 += 32) {  // ... and its tile that does
    const int64_t t = t0 + lane, u = t * step < s.n ? tile_units(w, s, static_cast<int>(t)) : 0;
    const int64_t cum = at + warp_scan(u * w.cut.nv, lane);
    const unsigned behind = __ballot_sync(0xffffffffu, cum > r.from);
    if (behind == 0) {
      at = __shfl_sync(0xffffffffu, cum, 31);
      continue;
    }
    const int k = __ffs(behind) - 1;
    const int64_t unit = __shfl_sync(0xffffffffu, u, k), begin = __shfl_sync(0xffffffffu, cum, k) - unit * w.cut.nv;
    r.tile = static_cast<int>(t0) + k;
    r.vh = static_cast<int>((r.from - begin) / unit);
    r.pos = begin + r.vh * unit;
    break;
  }
  return r;
}

// The first packed sequence behind b with new tokens, B or more if there is none: 128 looked at at a time by the warp, since
// others wait for what comes behind them and the waits are bounded.  Out of line: inlined in the
// walk it made the long chunk's kernel 2 % slower, without being called (1.30 vs 1.28 ms).
static __device__ __noinline__ int behind_empty(const int* cu, int N, int B, int b) {
  const int lane = threadIdx.x & 31;
  for (;;) {
    int n[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = b + 1 + 32 * k + lane;
      n[k] = 0;
      if (i < B) {
        const int from = min(max(cu[i], 0), N);
        n[k] = min(max(cu[i + 1], from), N) - from;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned some = __ballot_sync(0xffffffffu, n[k] > 0);
      if (some != 0) return b + 32 * k + __ffs(some);
    }
    b += 128;
    if (b >= B) return B;
  }
}

// The items of a CTA's stretch, one after another.
struct Walk {
  int64_t pos, from, to, stretch;  // this item on the line; the stretch
  int b, tile, vh;
  Seq s;
  int t0, t1, j0, n;
  bool pair;              // it fills two tiles
  int k0, k1;             // this CTA's blocks of the item: k0 .. k1 - 1
  int64_t end;            // the item's last block on the line

  __device__ __forceinline__ void set_tile(const Work& w) {
    t0 = tile * w.cut.step, t1 = min(s.n, t0 + w.cut.step);
    const Blocks k = blocks_of(w, s, t0, t1);
    j0 = k.j0, n = k.n;
    pair = t1 - t0 > w.cut.tile;
  }
  __device__ __forceinline__ void set_range() {
    end = pos + n - 1;
    k0 = from > pos ? static_cast<int>(min(static_cast<int64_t>(n), from - pos)) : 0;
    k1 = end >= to ? static_cast<int>(max(static_cast<int64_t>(0), to - pos)) : n;
  }
  // false: nothing to do
  __device__ __forceinline__ bool begin(const Work& w, const Plan& r) {
    if (r.b < 0) return false;
    stretch = r.stretch, from = r.from, to = r.to;
    pos = r.pos, b = r.b, tile = r.tile, vh = r.vh;
    s = seq_at(w.seqs, b);
    set_tile(w);
    set_range();
    return k0 < k1 || next(w);  // (the stretch may begin behind the item's last block)
  }
  // the next sequence with new tokens; false: there is none
  __device__ __forceinline__ bool next_sequence(const Work& w) {
    if (++b >= w.seqs.B) return false;
    s = seq_at(w.seqs, b);
    if (s.n == 0) {
      b = behind_empty(w.seqs.cu, w.seqs.N, w.seqs.B, b);
      if (b >= w.seqs.B) return false;
      s = seq_at(w.seqs, b);
    }
    return true;
  }
  // the next item with blocks in the stretch
  __device__ __forceinline__ bool next(const Work& w) {
    do {
      pos += static_cast<int64_t>(n) + w.cut.over;
      if (pos >= to) return false;
      if (++vh == w.cut.nv) {
        vh = 0;
        ++tile;
        if (static_cast<int64_t>(tile) * w.cut.step >= s.n) {
          tile = 0;
          if (!next_sequence(w)) return false;
        }
        set_tile(w);
      }
      set_range();
    } while (k0 >= k1);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == n; }
  __device__ __forceinline__ int slot(int p) const { return k0 > 0 ? 2 * p : 2 * p + 1; }
  // the CTAs whose stretches this item's blocks lie in, from this one on
  __device__ __forceinline__ int parts(int p) const { return static_cast<int>(end / stretch) - p + 1; }
};

// Where the outputs of a call go.
struct Out {
  void* O;
  float* lse;
  int64_t os[3], ls[2];
};

}  // namespace paged
}  // namespace fbd
