// What the tensor-core kernels of the attention over a paged cache share (tc_paged.cu, tc_paged_wide.cu).
#pragma once
#include <cuda_bf16.h>

#include "paged_launch.h"
#include "tmap.h"

namespace fbd {
namespace paged {

constexpr int BM = 128, BN = 128;
constexpr float kSlack = 256.f;  // the largest P
constexpr float kShare = .25f;   // ... and its share of the row's sum so far, where it is above 1
constexpr int kOut = 32 * 80;    // a warp's outputs on their way: 64 bytes of each row

// How K and V lie in the cache and in the ring.
struct Pages {
  int box;       // keys of a box
  int log;       // of the keys of a page to the base 2, -1 where they are no power of two
  int whole;     // a box takes all columns: its last coordinate is page * mul + head
  int mul;
  int sbo, slab; // bytes from eight keys to the next, from 64 columns to the next
};

// An item as the loading warp gives it to the others, through a ring in shared memory.
struct Item {
  int n;            // blocks b0 .. b0 + n - 1; 0: there are no more items
  int b0;
  int pair;         // two tiles see the same blocks; else both hold one tile's rows and take the blocks in turn
  int t0, t1;       // its tokens
  int start, len;   // of its sequence (paged.h)
  int last, first;  // the last key that every row sees, the first one
  int slot;         // of its part of a shared item, -1: it is whole
  int b, batch, row0, vh, kvh, pad;
  // some row does not see some key of the block (of `keys` keys)
  __device__ __forceinline__ bool hides(int kb, int keys = BN) const { return kb * keys + keys - 1 > last || kb * keys < first; }
  __device__ __forceinline__ int count(int m) const { return pair ? n : (n + 1 - m) / 2; }  // blocks of tile m
};

// The ring's entries of an item: two tiles over the same blocks: K_0 V_0 K_1 V_1 ...; one tile whose blocks
// go to both in turn: K_0 K_1 V_0 K_2 V_1 K_3 ...; 2 n in all.
struct Order {
  int base, n;
  bool pair;
  __device__ __forceinline__ int block(int m, int j) const { return pair ? j : 2 * j + m; }
  __device__ __forceinline__ int V(int i) const {
    return pair ? base + 2 * i + 1 : base + min(n, 2) + i + min(i, max(n - 2, 0));
  }
  __device__ __forceinline__ int K(int i) const { return pair ? base + 2 * i : i < 2 ? base + i : V(i - 2) + 1; }
};

// Values that were made 0 for the rows that do not see them, added to a row that does (`o` or `part`, its
// first d columns): one by one from the cache.
static __device__ __noinline__ void add_spoilt(const Work& w, const Item& it, int first, int last, const __nv_bfloat16* V, int64_t s0,
                                        int64_t s2, int d, __nv_bfloat16* o, float* part, int keys = BN) {
  for (int i = 0; i < it.n; ++i) {
    const int k0 = (it.b0 + i) * keys;
    if (!it.hides(it.b0 + i, keys)) continue;
    for (int k = max(k0, first); k <= min(k0 + keys - 1, last); ++k) {
      const int pg = page_at(w.seqs, it.b, k / w.seqs.page);
      if (pg < 0) continue;
      const __nv_bfloat16* v = V + pg * s0 + static_cast<int64_t>(k % w.seqs.page) * s2;
      for (int x = 0; x < d; ++x) {
        const float y = __bfloat162float(v[x]);
        if (isfinite(y)) continue;
        if (part != nullptr) part[x] += y;
        else o[x] = __float2bfloat16(__bfloat162float(o[x]) + y);
      }
    }
  }
}

// A lane's box of a run of keys (an entry of the ring, or two of the same keys): its place in the run, the page and the
// slot there that it reads (page < 0: zeros), and of all the warp's the 16-key runs without a page.
struct Box {
  int page, slot;
  uint32_t hidden;
};
// `keys` keys from k0 on, `per` boxes of them, this lane's the g-th.
__device__ __forceinline__ Box box_at(const Work& w, const Pages& pg, const Seq& s, int b, int k0, int g, int per) {
  const int key = k0 + g * pg.box, e = pg.log >= 0 ? key >> pg.log : key / w.seqs.page;
  const bool mine = g < per && key < s.len;
  Box x;
  x.page = mine ? page_at(w.seqs, b, e) : -1;
  x.slot = x.page < 0 ? 0 : key - e * w.seqs.page;
  x.hidden = __reduce_or_sync(0xffffffffu, mine && x.page < 0 ? ((1u << (pg.box / 16)) - 1u) << (g * (pg.box / 16)) : 0u);
  return x;
}
// The warp's copies (one lane's after another's).
__device__ __forceinline__ void load_box(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, const Pages& pg, const Box& x, int g,
                                         int per, int slab, int kvh) {
  if (g >= per) return;
  dst += (g * pg.box >> 3) * pg.sbo + slab * pg.slab;
  if (pg.whole)
    ptx::tma_load_5d(dst, map, bar, 0, 0, 0, x.slot >> 3, x.page < 0 ? -1 : x.page * pg.mul + kvh);
  else
    ptx::tma_load_4d(dst, map, bar, slab * 64, x.slot, kvh, x.page);
}

// 64 bytes of each live row of a warp to `to`, its own row's address, through `stage` (kOut bytes of the warp's own):
// four threads write 64 bytes of a row.
__device__ __forceinline__ void put_rows(uint8_t* stage, const uint32_t (&x)[16], uint8_t* to, bool live) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(stage + lane * 80 + u * 16) = make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
  __syncwarp();
  const unsigned rows = __ballot_sync(0xffffffffu, live);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = u * 8 + (lane >> 2);
    uint8_t* at = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), row));
    const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 80 + (lane & 3) * 16);
    if (rows >> row & 1) *reinterpret_cast<uint4*>(at + (lane & 3) * 16) = v;
  }
}

// Values of `keys` keys in shared memory, by a warp: 0 behind the `held` first keys, and where they are not finite;
// true if some of this lane's were.
__device__ __forceinline__ bool hide_values(uint8_t* V, int keys, int held, int slabs, const Pages& pg) {
  bool some = false;
  for (int r = threadIdx.x & 31; r < keys; r += 32) {
    uint8_t* row = V + (r >> 3) * pg.sbo + (r & 7) * 128;
    for (int u = 0; u < slabs; ++u, row += pg.slab) {
      uint4* at = reinterpret_cast<uint4*>(row);  // (its 16-byte pieces in another order)
      if (r >= held) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) at[ch ^ (r & 7)] = make_uint4(0, 0, 0, 0);
        continue;
      }
      uint32_t top = 0;  // an exponent of ones carries into the sign's place
      uint4 x[8];
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) x[ch] = at[ch ^ (r & 7)];
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
        top |= ((x[ch].x & 0x7f807f80u) + 0x00800080u) | ((x[ch].y & 0x7f807f80u) + 0x00800080u) |
               ((x[ch].z & 0x7f807f80u) + 0x00800080u) | ((x[ch].w & 0x7f807f80u) + 0x00800080u);
      if ((top & 0x80008000u) == 0) continue;
      some = true;
      uint16_t* e = reinterpret_cast<uint16_t*>(row);
      for (int k = 0; k < 64; ++k)
        if ((e[k] & 0x7f80u) == 0x7f80u) e[k] = 0;
    }
  }
  return some;
}

// Tensor maps of Q (a tile's tokens and heads; mq may be null), K and V in entries of `keys` keys and `slabs` slabs of 64
// columns.
inline bool make_maps(const PagedArgs& a, const Cut& k, int keys, int slabs, void* mq, void* mk, void* mv, Pages& pg) {
  const bool none = a.seqs.pages == 0;  // no key anywhere: a tensor that is never read
  const int64_t q_dims[5] = {a.d, k.gt, a.seqs.N, k.nv, a.seqs.cu != nullptr ? 1 : a.seqs.B};
  const int64_t q_str[4] = {a.qs[1], a.qs[2], a.qs[1] * k.gt, a.qs[0]};
  const int q_box[5] = {64, k.gt, k.tile, 1, 1};
  if (mq != nullptr && !make_tmap_view(mq, a.Q, 5, q_dims, q_str, q_box)) return false;
  pg.log = -1;
  for (int k = 4; k <= 20; ++k)
    if (a.seqs.page == 1 << k) pg.log = k;
  pg.box = keys;  // as many keys as divide a page's
  while (a.seqs.page % pg.box != 0) pg.box /= 2;
  // All columns in a box: of whole slabs, and pages a multiple of the heads' stride apart (K and V alike, and
  // within a coordinate).
  const int64_t pages = none ? 1 : a.seqs.pages, one = a.Hkv == 1 ? 1 : 0;
  const int64_t k_mul = one ? 1 : pages == 1 ? 0 : a.ks[0] / a.ks[1], v_mul = one ? 1 : pages == 1 ? 0 : a.vs[0] / a.vs[1];
  const int64_t heads = (pages - 1) * k_mul + a.Hkv;
  pg.whole = a.d % 64 == 0 && !none && k_mul == v_mul && heads < (int64_t(1) << 31) &&
             (one || pages == 1 || (a.ks[0] % a.ks[1] == 0 && a.vs[0] % a.vs[1] == 0));
  pg.mul = static_cast<int>(k_mul);
  const void *K = none ? a.Q : a.K, *V = none ? a.Q : a.V;
  bool made;
  if (pg.whole) {
    pg.slab = 1024, pg.sbo = slabs * 1024;
    const int64_t dims[5] = {64, 8, a.d / 64, a.seqs.page / 8, heads};
    const int64_t k_str[4] = {a.ks[2], 64, 8 * a.ks[2], one ? a.ks[0] : a.ks[1]}, v_str[4] = {a.vs[2], 64, 8 * a.vs[2], one ? a.vs[0] : a.vs[1]};
    const int boxes[5] = {64, 8, a.d / 64, pg.box / 8, 1};
    made = make_tmap_view(mk, K, 5, dims, k_str, boxes) && make_tmap_view(mv, V, 5, dims, v_str, boxes);
  } else {
    pg.slab = keys * 128, pg.sbo = 1024;
    const int64_t dims[4] = {a.d, a.seqs.page, a.Hkv, pages};
    const int64_t k_str[3] = {a.ks[2], a.ks[1], a.ks[0]}, v_str[3] = {a.vs[2], a.vs[1], a.vs[0]};
    const int boxes[4] = {64, pg.box, 1, 1};
    made = make_tmap_view(mk, K, 4, dims, k_str, boxes) && make_tmap_view(mv, V, 4, dims, v_str, boxes);
  }
  return made;
}

}  // namespace paged
}  // namespace fbd
