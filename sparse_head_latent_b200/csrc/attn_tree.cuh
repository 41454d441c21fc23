// attn_tree.cuh -- attention of a tree of drafted tokens over a paged latent
// cache, absorbed form (sm_100a).
//
// Sequence b holds cache_len[b] committed positions and n_nodes[b] drafted
// ones behind them; position t lives in row t mod page of page
// block_table[b][t / page]. Node j sits at position cache_len[b] + j and sees
// the committed positions, itself, and the nodes above it in the tree:
//   z_t      = scale [q_abs | q_pe] . [c_t | k_pe_t]     (576 wide)
//   o_lat    = sum_t softmax(z)_t c_t
// per (node, head); q_abs = q_nope W_UK before, attn = W_UV o_lat after it.
#pragma once

#include "ptx.cuh"

namespace mla {

constexpr int kTreeMax = 64;  // nodes per sequence: one bit each

struct TreeParams {
  int B, N, H;
  int num_pages, page_shift, table_width;
  float scale_log2;              // softmax scale * log2(e)
  const int32_t* table;          // [B][table_width]
  const int32_t* cache_len;      // [B]
  const int32_t* n_nodes;        // [B], or nullptr: N each
  const int32_t* parents;        // [B][N], or nullptr: a chain
  const __nv_bfloat16* qabs;     // [B*N][H][512]
  const __nv_bfloat16* q;        // [B*N][H][192] (rope at 128..191)
  const __nv_bfloat16* kv;       // [num_pages * page][512]
  const __nv_bfloat16* pe;       // [num_pages * page][64]
  __nv_bfloat16* olat;           // [B*N][H][512]
  int* err;
};

// Lengths of sequence b: committed positions and nodes. A sequence whose
// positions do not fit its row of the table has no nodes (error 402).
__device__ __forceinline__ void tree_lengths(const TreeParams& p, int b, int& len, int& nodes) {
  len = __ldg(p.cache_len + b);
  nodes = p.n_nodes ? min(max(__ldg(p.n_nodes + b), 0), p.N) : p.N;
  if (len < 0 || len + static_cast<int64_t>(nodes) > (static_cast<int64_t>(p.table_width) << p.page_shift)) {
    atomicCAS(p.err, 0, kErrLength);
    len = nodes = 0;
  }
}

constexpr int kTreeKeys = 32;
constexpr int kTreeWarps = 8;

// One warp per (node, head), eight heads of a node per block; the block
// stages 32 positions at a time.
__global__ void __launch_bounds__(32 * kTreeWarps)
tree_attn_kernel(const TreeParams p) {
  __shared__ __align__(16) __nv_bfloat16 keys[kTreeKeys][576 + 8];
  __shared__ __nv_bfloat16 qs[kTreeWarps][576];
  const int hg = (p.H + kTreeWarps - 1) / kTreeWarps;
  const int node_row = blockIdx.x / hg, b = node_row / p.N, j = node_row % p.N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (blockIdx.x % hg) * kTreeWarps + warp;
  int len, nodes;
  tree_lengths(p, b, len, nodes);
  const int64_t qrow = static_cast<int64_t>(node_row) * p.H + min(h, p.H - 1);
  float acc[16], m = -INFINITY, l = 0.f;
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  if (j < nodes) {
    uint64_t sees = 1ull << j;
    if (p.parents) {
      int k = j;
      while (true) {
        const int up = __ldg(p.parents + static_cast<int64_t>(b) * p.N + k);
        if (up < 0 || up >= k) break;
        sees |= 1ull << up;
        k = up;
      }
    } else {
      sees |= (1ull << j) - 1;
    }
    for (int d = lane; d < 576; d += 32)
      qs[warp][d] = d < 512 ? p.qabs[qrow * 512 + d] : p.q[qrow * 192 + 128 + d - 512];
    const int T = len + nodes;
    for (int t0 = 0; t0 < T; t0 += kTreeKeys) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTreeKeys * 72; i += 32 * kTreeWarps) {
        const int r = i / 72, c = i % 72, t = t0 + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t < T) {
          const int page = __ldg(p.table + static_cast<int64_t>(b) * p.table_width + (t >> p.page_shift));
          if (page >= 0 && page < p.num_pages) {
            const int64_t row = (static_cast<int64_t>(page) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
            v = __ldg(reinterpret_cast<const uint4*>(c < 64 ? p.kv + row * 512 + c * 8 : p.pe + row * 64 + (c - 64) * 8));
          } else if (c == 0) {
            atomicCAS(p.err, 0, kErrPage);
          }
        }
        *reinterpret_cast<uint4*>(&keys[r][c * 8]) = v;
      }
      __syncthreads();
      const int t = t0 + lane;
      const bool seen = t < len || (t < T && ((sees >> (t - len)) & 1));
      float z = 0.f;
      for (int d = 0; d < 576; d += 2) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&keys[lane][d]));
        z = fmaf(__bfloat162float(qs[warp][d]), f.x, fmaf(__bfloat162float(qs[warp][d + 1]), f.y, z));
      }
      z = seen ? z * p.scale_log2 : -INFINITY;
      float top = z;
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m_new = fmaxf(m, top);
      if (m_new == -INFINITY) continue;
      const float alpha = exp2f(m - m_new), w = seen ? exp2f(z - m_new) : 0.f;
      m = m_new;
      l = l * alpha + w;
      for (int i = 0; i < 16; ++i) acc[i] *= alpha;
      for (int k = 0; k < kTreeKeys; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (!__shfl_sync(0xffffffffu, static_cast<int>(seen), k)) continue;
        for (int i = 0; i < 8; ++i) {
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&keys[k][lane * 16 + 2 * i]));
          acc[2 * i] = fmaf(wk, f.x, acc[2 * i]);
          acc[2 * i + 1] = fmaf(wk, f.y, acc[2 * i + 1]);
        }
      }
    }
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  }
  if (h >= p.H) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.olat + qrow * 512 + lane * 16);
  for (int i = 0; i < 8; ++i) dst[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
}

}  // namespace mla
