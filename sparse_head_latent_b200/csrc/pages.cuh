// pages.cuh -- upkeep of a paged latent cache (sm_100a): the rows of an
// accepted path moved together, pages copied. Both only move bytes, for every
// layer of the cache in one launch; memory bounds them, and the launch when
// there is one row.
#pragma once

#include "ptx.cuh"

namespace mla {

constexpr int kRowPieces = 72;  // 16-byte pieces of a cached position: 64 latent, 8 rope

// Address of piece c of cache row r.
__device__ __forceinline__ uint4* cache_piece(uint4* kv, uint4* pe, int64_t r, int c) {
  return c < 64 ? kv + r * 64 + c : pe + r * 8 + (c - 64);
}

struct CompactParams {
  uint4* kv;                  // [layers][num_pages * page][512] bf16
  uint4* pe;                  // [layers][num_pages * page][64]
  int layers, num_pages, page_shift, table_width;
  const int32_t* table;       // [B][table_width]
  const int32_t* cache_len;   // [B]
  const int32_t* accepted;    // [B][width]
  const int32_t* counts;      // [B]
  int width;
  int* err;
};


// Block (b, LAYERS layers): row cache_len + accepted[i] of the sequence to row
// cache_len + i, for i < counts[b]. Sources and destinations overlap (a
// destination can be a later source), so the block reads all its rows into
// registers, waits for all its threads, and only then writes; no other block
// touches this sequence's rows of these layers. SIDE rows are moved side by side,
// and a thread holds PER of a layer. The rows are found one per thread, through
// two loads in a row (length, count and node, then page), and passed on in shared
// memory. 64 sequences, 60 layers, up to 16 rows each, 71 MB moved: 15.7 us; up
// to 32 rows, 141 MB: 27.3. With every thread looking for its rows itself 20.5
// and 108.
template <int SIDE, int PER, int LAYERS>
__global__ void __launch_bounds__(kRowPieces * SIDE)
cache_compact_kernel(const CompactParams p) {
  __shared__ int from[SIDE * PER], to[SIDE * PER];
  const int b = blockIdx.x, i = static_cast<int>(threadIdx.x);
  const int node = i < p.width ? __ldg(p.accepted + static_cast<int64_t>(b) * p.width + i) : -1;
  const int count = min(__ldg(p.counts + b), p.width);
  const int64_t len = __ldg(p.cache_len + b);
  if (count <= 0) return;
  if (i < count) {
    // cache row of position t, or -1 when it lies outside the table or the cache
    auto place = [&](int64_t t) -> int {
      const int64_t at = t >> p.page_shift;
      if (t < 0 || at >= p.table_width) return -1;
      const int page = __ldg(p.table + static_cast<int64_t>(b) * p.table_width + at);
      if (page < 0 || page >= p.num_pages) return -1;
      return (page << p.page_shift) + static_cast<int>(t & ((1 << p.page_shift) - 1));
    };
    const int f = node < 0 ? -1 : place(len + node), t = place(len + i);
    if (f < 0 || t < 0) atomicCAS(p.err, 0, kErrPage);
    from[i] = f;
    to[i] = f < 0 || f == t ? -1 : t;  // f == t: already there
  }
  __syncthreads();
  const int64_t rows = static_cast<int64_t>(p.num_pages) << p.page_shift;
  const int layer0 = static_cast<int>(blockIdx.y) * LAYERS;
  const int c = i % kRowPieces, r0 = i / kRowPieces;
  uint4 v[PER][LAYERS];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int r = r0 + k * SIDE;
    if (r >= count || to[r] < 0) continue;
#pragma unroll
    for (int l = 0; l < LAYERS; ++l)
      if (layer0 + l < p.layers) v[k][l] = *cache_piece(p.kv, p.pe, (layer0 + l) * rows + from[r], c);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int r = r0 + k * SIDE;
    if (r >= count || to[r] < 0) continue;
#pragma unroll
    for (int l = 0; l < LAYERS; ++l)
      if (layer0 + l < p.layers) *cache_piece(p.kv, p.pe, (layer0 + l) * rows + to[r], c) = v[k][l];
  }
}

// Pairs of pages by value: a launch carries this many (4 KB of parameters).
constexpr int kCopyPairs = 480;
struct PagePairs {
  int src[kCopyPairs], dst[kCopyPairs];
};

constexpr int kCopyThreads = 256;
constexpr int kCopyPer = 4;  // 16-byte pieces a thread has in flight

// Block (piece of a page, pair, layer): the page's latent rows, then its rope
// rows, as one run of 72 * page pieces. 48 pairs, 60 layers, pages of 64, 425 MB
// moved: 58 us, 7.3 TB/s (above the rate of a plain copy: part of it stays in L2).
__global__ void __launch_bounds__(kCopyThreads)
cache_copy_kernel(const __grid_constant__ PagePairs pp, uint4* kv, uint4* pe, int num_pages, int page) {
  const int64_t s = pp.src[blockIdx.y], d = pp.dst[blockIdx.y];
  const int64_t layer = blockIdx.z;
  uint4* lk = kv + layer * num_pages * page * 64;
  uint4* lp = pe + layer * num_pages * page * 8;
  const int64_t np = int64_t(page) * 8, nk = np * 8, n = nk + np;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kCopyThreads * kCopyPer + threadIdx.x;
  uint4 v[kCopyPer];
#pragma unroll
  for (int k = 0; k < kCopyPer; ++k) {
    const int64_t i = i0 + k * kCopyThreads;
    if (i < n) v[k] = i < nk ? lk[s * nk + i] : lp[s * np + (i - nk)];
  }
#pragma unroll
  for (int k = 0; k < kCopyPer; ++k) {
    const int64_t i = i0 + k * kCopyThreads;
    if (i < n) {
      if (i < nk) lk[d * nk + i] = v[k];
      else lp[d * np + (i - nk)] = v[k];
    }
  }
}

}  // namespace mla
