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
//
// All (node, head) rows of a sequence meet the same keys, so they are the rows
// of one matrix product: tiles of 128 rows (H = 128: one node a tile) against
// blocks of 128 keys. Work item: one CTA pair per run of consecutive (tile,
// block) units; the units of all sequences, tile after tile, are cut into
// equal shares, one per resident pair, so that ragged lengths, one long
// sequence and many short ones all fill the machine. A tile that several pairs
// share is joined by tree_combine_kernel.
//
// Shape of the products. A pair UMMA with M = 128 gives each CTA 64 rows and
// uses all 128 lanes of its tensor memory: lanes 0..63 hold columns [0, N/2) of
// rows 0..63, lanes 64..127 columns [N/2, N). O (64 rows x 512 fp32) then takes
// 256 of the 512 columns, where 128 rows in one CTA would take all of them and
// leave none for S. Rates of the tensor core alone, clk per block of 128 keys
// (full rate in brackets): Q.K^T 1161 (1152), P.V 1037 (1024), both 2190.
//
// A block is 2.2k clk of tensor core, but 136 KB per CTA if Q.K^T's keys and
// P.V's values are loaded apart, and L2 -> SM then sets the pace (4.1k clk a
// block; 2.9k with half the bytes). So a block is kept in place: for Q.K^T a
// CTA holds its own 64 of the block's keys, all 512 latent values of each, as
// four 16 KB groups of 128 values; for P.V it needs all 128 keys, its own half
// of each 256 values. The two meet: group i = 2 h + r of CTA r is already the
// values [256 h + 128 r, + 128) of its own keys. The other two groups it is
// done with once Q.K^T has read them, and loads them again with the other keys'
// values of its half. Group 2 h + k then holds, in both CTAs, keys [64 k, + 64)
// of the block, values of half h, and each CTA has loaded 13 chunks of 64 values
// instead of 17. The price is that groups stay taken through the softmax: ten
// fit, two and a half blocks, because six of Q's nine chunks live in tensor
// memory (next to O and one S; Q.K^T(j + 1) waits until S(j) has been loaded,
// which P.V(j - 1) covers). Those six travel through the ring, too: three groups
// in front of a run's first block, which the softmax warps copy.
//
// Roles (352 threads per CTA): warps 0 and 10 producers, of keys and of values
// (warp 0 also walks the share and publishes its runs); warp 1 of the leader
// issues the UMMAs; warps 2..9 softmax: four threads per row, one for each
// quarter of the block's keys, agree on the running maximum through shared
// memory.
//
// Measured: 8192 rows against 32768 keys 362 us, 1.61 PFLOP/s (tensor core);
// 64 sequences of 128 rows and 30000 to 32768 keys 449 us, 5.2 TB/s of cache (L2
// -> SM and HBM); 98 tiles of 4 to 63 blocks 105 us, half of it tensor core: a
// run costs about three blocks before and after its products.
#pragma once

#include "gemm2.cuh"
#include "ptx.cuh"

namespace mla {

constexpr int kTreeMax = 64;        // nodes per sequence: one bit each
constexpr int kTreeRows = 128;      // rows of a tile
constexpr int kTreeBlock = 128;     // keys of a block
constexpr int kTreeMaxPairs = 74;   // pairs a launch uses at most (148 SMs); the workspace is sized for them
constexpr int kTreeThreads = 352;
// What a tile costs a pair besides its blocks, in blocks: Q's loads, the first
// products with nothing before them, the result. Where there are more tiles than
// pairs the shares count it: 98 tiles of 4 to 63 blocks took 145 us in shares of
// equal blocks, 120, 118, 120 and 125 with 2, 3, 4 and 7 added. With fewer tiles
// every pair has about one run, and counting it would take blocks from none.
constexpr int kTreeRunCost = 3;
constexpr int kTreeSlotFloats = kTreeRows * 512;  // one partial tile

struct TreeParams {
  int B, N, H;
  int num_pages, page_shift, table_width;
  int box_shift;                 // log2 of the keys per TMA box: min(page, 64)
  float scale_log2;              // softmax scale * log2(e)
  const uint4* kv;               // the cache's latents again, 64 pieces a row
  const int32_t* table;          // [B][table_width]
  const int32_t* cache_len;      // [B]
  const int32_t* n_nodes;        // [B], or nullptr: N each
  const int32_t* parents;        // [B][N], or nullptr: a chain
  const float* v_scale;          // [2 H][4], or nullptr: row 2 h + 1 multiplies the four 128s of head h's o_lat
  __nv_bfloat16* olat;           // [B*N][H][512]
  int64_t* ustart;               // [B + 2] first unit of each sequence, their number, and what a tile adds to its blocks
  float* part_o;                 // [2 pairs][128 value quads][128 rows][4] unnormalised partial tiles
  float2* part_ml;               // [2 pairs][128 rows] (max in the scaled log2 domain, sum)
  int most_blocks;               // of a tile whose keys are loaded: all, fewer by the test hook only
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

__device__ __forceinline__ void tree_extent(const TreeParams& p, int len, int nodes, int& tiles, int& blocks) {
  tiles = (nodes * p.H + kTreeRows - 1) / kTreeRows;
  blocks = nodes > 0 ? (len + nodes + kTreeBlock - 1) / kTreeBlock : 0;
}

// A run of a pair's work: blocks [j0, j1) of one tile.
struct TreeRun {
  int b, tile, j0, j1;
  int len, nodes, blocks;  // of sequence b
  int flags;               // 1: the pair's first run, 2: another one follows
};

// Where a pair stands in its share of the units.
struct TreeWork {
  int64_t left;                   // units still to walk, without the open tile's own
  int b, tile, j;                 // where the next run begins
  int len, nodes, tiles, blocks;  // of sequence b
  int first, extra;               // units of a tile besides its blocks
  __device__ __forceinline__ TreeRun next(const TreeParams& p) {
    while (tile >= tiles) {
      tree_lengths(p, ++b, len, nodes);
      tree_extent(p, len, nodes, tiles, blocks);
      tile = 0;
    }
    TreeRun r;
    r.b = b;
    r.tile = tile++;
    r.j0 = j;
    r.j1 = left < blocks - j ? j + static_cast<int>(left) : blocks;
    r.len = len;
    r.nodes = nodes;
    r.blocks = blocks;
    left -= r.j1 - j + extra;
    r.flags = first | (left > 0 ? 2 : 0);
    first = 0;
    j = 0;
    return r;
  }
};

// First units of the shares of `pair` and of the next: equal, the first
// units % pairs of them one longer. One division, of 64 bits: a few hundred
// clk, on the way to a block's first load.
__device__ __forceinline__ void tree_share(int64_t units, int pair, int pairs, int64_t& u0, int64_t& u1) {
  const int64_t each = units / pairs, more = units - each * pairs;
  u0 = each * pair + (pair < more ? pair : more);
  u1 = u0 + each + (pair < more ? 1 : 0);
}

struct TreeSmem {
  static constexpr int CHUNK = 8192;               // [64 keys or rows x 64] bf16
  static constexpr int GROUP = 2 * CHUNK;
  static constexpr int GROUPS = 10;
  static constexpr int ROPES = 2;                  // blocks whose rope chunks fit
  static constexpr int Q_TMEM = 6;                 // chunks of Q in tensor memory, the first of the nine
  static constexpr int Q_GROUPS = Q_TMEM / 2;      // as groups of the ring
  static constexpr int Q_CHUNKS = 9 - Q_TMEM;      // and in shared memory
  static constexpr int RING = 0;
  static constexpr int ROPE = RING + GROUPS * GROUP;
  static constexpr int Q = ROPE + ROPES * CHUNK;
  static constexpr int P = Q + Q_CHUNKS * CHUNK;   // two [64 rows x 64 keys] chunks
  static constexpr int XCHG = P + 2 * CHUNK;       // [2][4][64] floats
  static constexpr int BARS = XCHG + 2 * 4 * 64 * 4;
  static constexpr int START = BARS + 400;         // where the share begins: sequence, tile, block, extra units
  static constexpr int RUNS = BARS + 416;          // four TreeRuns, published by the producer of keys
  static constexpr int BYTES = RUNS + 4 * 32;
};
static_assert(TreeSmem::BYTES <= 232448, "shared memory per CTA");

// Barriers; (L): only the leader's copy is used, by both CTAs.
enum : int {
  kTreeKFull = 0,                               // (L) per group: the own keys' values landed in both CTAs
  kTreeVFull = kTreeKFull + TreeSmem::GROUPS,   // (L) per group: the other keys' values landed in the CTA that reloads it
  kTreeEmpty = kTreeVFull + TreeSmem::GROUPS,   // per group: the P.V that read it is done
  // Q.K^T of a block is done; one barrier for even and one for odd blocks, since
  // the next block's may be done before the producer looks for this one's.
  kTreeSFull = kTreeEmpty + TreeSmem::GROUPS,
  kTreeSFree = kTreeSFull + 2,                  // (L) S is in the softmax warps' registers (sixteen warps)
  kTreePVDone,                                  // P.V of a block is done
  kTreeRopeFull,                                // (L) per rope slot: the chunk landed in both CTAs
  kTreeQFull = kTreeRopeFull + TreeSmem::ROPES,                                   // (L) Q's shared-memory part landed in both CTAs
  kTreeRun,                                     // a run's description is in the ring; two, taken in turn
  kTreeQGroups = kTreeRun + 2,                  // the three groups of its tensor-memory part landed in this CTA; two,
                                                // taken in turn, since a run of one block is requested two runs ahead
  kTreeQReady = kTreeQGroups + 2,                                // (L) they are in tensor memory (sixteen warps)
  kTreePFull,                                   // (L) P of both CTAs is written (sixteen warps)
  kTreeTail,                                    // the reloaded values of a block with drafted keys landed in this
                                                // CTA; two, taken in turn
  kTreeXchg = kTreeTail + 2,                    // per 32 rows: their four softmax warps have written their values
  kTreeOut = kTreeXchg + 2,                     // the eight softmax warps of this CTA meet
  kTreeDrain,
  kTreeBars
};
static_assert(8 * kTreeBars + 8 <= 400 && sizeof(TreeRun) == 32, "layout behind the barriers");

constexpr uint32_t kTreeColS = 256;  // S; O at 0 and 128
constexpr uint32_t kTreeColQ = 320;  // Q's first six chunks, 32 columns each

// Nodes that node j of sequence b sees, as bits (itself included); every lane
// of the warp asks for its own j. The parents of nodes `lane` and `lane + 32`
// are in registers; six rounds double the distance looked up.
__device__ __forceinline__ uint64_t tree_ancestors(const TreeParams& p, int b, int j) {
  if (p.parents == nullptr) return j < kTreeMax ? (j == 63 ? ~0ull : (2ull << j) - 1) : 0ull;
  const int lane = static_cast<int>(lane_id());
  uint64_t sees[2];
  int up[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = lane + 32 * i;
    sees[i] = 1ull << k;
    const int v = k < p.N ? __ldg(p.parents + static_cast<int64_t>(b) * p.N + k) : -1;
    up[i] = v >= 0 && v < k ? v : -1;
  }
#pragma unroll 1
  for (int round = 0; round < 6; ++round) {
    uint64_t s2[2];
    int u2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int from = max(up[i], 0);
      const uint64_t a = __shfl_sync(0xffffffffu, sees[0], from & 31), c = __shfl_sync(0xffffffffu, sees[1], from & 31);
      const int d = __shfl_sync(0xffffffffu, up[0], from & 31), e = __shfl_sync(0xffffffffu, up[1], from & 31);
      s2[i] = up[i] < 0 ? 0ull : from < 32 ? a : c;
      u2[i] = up[i] < 0 ? -1 : from < 32 ? d : e;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sees[i] |= s2[i];
      up[i] = u2[i];
    }
  }
  const uint64_t a = __shfl_sync(0xffffffffu, sees[0], j & 31), c = __shfl_sync(0xffffffffu, sees[1], j & 31);
  return j < 32 ? a : j < kTreeMax ? c : 0ull;
}

// Which of the 32 keys from position t0 on a row sees, as bits.
__device__ __forceinline__ uint32_t tree_keep(int64_t t0, int len, uint64_t sees) {
  const int64_t d = t0 - len;
  if (d >= kTreeMax) return 0u;
  if (d >= 0) return static_cast<uint32_t>(sees >> d);
  if (d <= -32) return ~0u;
  return static_cast<uint32_t>(sees << -d) | ((1u << -d) - 1u);
}

// Whether one of a sequence's positions t0 + i below `total`, i in `which`, has a
// latent value that is not finite; `table` is the sequence's own row. For scores of
// -inf only: out of line, one thread.
__device__ __noinline__ bool tree_latent_not_finite(const uint4* kv, const int32_t* table, int page_shift, int num_pages,
                                                    int64_t t0, int total, uint32_t which) {
  for (; which != 0u; which &= which - 1u) {
    const int64_t t = t0 + __ffs(static_cast<int>(which)) - 1;
    if (t >= total) return false;  // rows of nodes that are not there look behind the last position
    const int page = __ldg(table + (t >> page_shift));
    if (page < 0 || page >= num_pages) continue;
    const uint4* row = kv + ((static_cast<int64_t>(page) << page_shift) + (t & ((1 << page_shift) - 1))) * 64;
    for (int i = 0; i < 64; ++i) {
      const uint4 v = row[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      for (int e = 0; e < 4; ++e)
        if ((w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u) return true;
    }
  }
  return false;
}

__global__ void __launch_bounds__(kTreeThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_pe,
                 const __grid_constant__ CUtensorMap tm_qabs, const __grid_constant__ CUtensorMap tm_q,
                 const TreeParams p) {
  using S = TreeSmem;
  // Every byte is in use, so the swizzle's 1024-byte alignment is the base's
  // own (dynamic shared memory starts there without static shared memory).
  extern __shared__ __align__(1024) uint8_t smem[];
  if (blockDim.x != kTreeThreads || (smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kErrGeometry);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kTreeBars);
  int* abort_word = reinterpret_cast<int*>(tmem_slot + 1);
  int* start = reinterpret_cast<int*>(smem + S::START);
  TreeRun* run_ring = reinterpret_cast<TreeRun*>(smem + S::RUNS);
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;

  if (threadIdx.x >= 64 && threadIdx.x < 64 + kTreeBars) {
    const int i = static_cast<int>(threadIdx.x) - 64;
    const bool both = i == kTreeSFree || i == kTreePFull || i == kTreeQReady;
    mbar_init(bar(i), both ? 16 : i == kTreeOut ? 8 : i == kTreeXchg || i == kTreeXchg + 1 ? 4 : 1);
    if (i == 0) *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_kv);
    prefetch_tmap(&tm_pe);
    prefetch_tmap(&tm_qabs);
    prefetch_tmap(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  // The share: units of all sequences, scanned by the whole CTA, each thread
  // a run of sequences.
  TreeWork work;
  {
    int64_t* sums = reinterpret_cast<int64_t*>(smem + S::XCHG);  // per warp: blocks, tiles
    const int per = (p.B + kTreeThreads - 1) / kTreeThreads;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    int64_t blocks_mine = 0;
    int tiles_mine = 0;  // 2^28 in all at most
    for (int b = b0; b < b1; ++b) {
      int len, nodes, tiles, blocks;
      tree_lengths(p, b, len, nodes);
      tree_extent(p, len, nodes, tiles, blocks);
      blocks_mine += static_cast<int64_t>(tiles) * blocks;
      tiles_mine += tiles;
    }
    int64_t blocks_to = blocks_mine;
    int tiles_to = tiles_mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, blocks_to, o);
      const int w = __shfl_up_sync(0xffffffffu, tiles_to, o);
      if (lane >= o) blocks_to += v, tiles_to += w;
    }
    if (lane == 31) sums[2 * warp] = blocks_to, sums[2 * warp + 1] = tiles_to;
    __syncthreads();
    int64_t total = 0, tiles_all = 0;
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      if (w < warp) blocks_to += sums[2 * w], tiles_to += static_cast<int>(sums[2 * w + 1]);
      total += sums[2 * w];
      tiles_all += sums[2 * w + 1];
    }
    const int extra = tiles_all > pairs ? kTreeRunCost : 0;
    total += extra * tiles_all;
    int64_t at = blocks_to - blocks_mine + static_cast<int64_t>(extra) * (tiles_to - tiles_mine);
    int64_t u0, u1;
    tree_share(total, pair, pairs, u0, u1);
    const bool mark = blockIdx.x == 0, here = u0 >= at && u0 < at + blocks_mine + static_cast<int64_t>(extra) * tiles_mine;
    if (mark || here) {
      for (int b = b0; b < b1; ++b) {
        int len, nodes, tiles, blocks;
        tree_lengths(p, b, len, nodes);
        tree_extent(p, len, nodes, tiles, blocks);
        const int64_t units = static_cast<int64_t>(tiles) * (blocks + extra);
        if (mark) p.ustart[b] = at;
        if (u0 >= at && u0 < at + units) {
          const int64_t tile = (u0 - at) / (blocks + extra);
          const int off = static_cast<int>(u0 - at - tile * (blocks + extra));
          start[0] = b;
          start[1] = static_cast<int>(tile);
          start[2] = max(0, off - extra);
          start[3] = max(0, extra - off);  // of the first run's own units
        }
        at += units;
      }
    }
    if (mark && threadIdx.x == 0) {
      p.ustart[p.B] = total;
      p.ustart[p.B + 1] = extra;
    }
    work.left = u1 - u0;
    work.extra = extra;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  griddep_launch();
  if (work.left > 0) work.left -= start[3];
  const bool busy = work.left > 0;  // the pair has work at all
  const uint32_t tmem = *tmem_slot;
  const Abort ab{abort_word, p.err};

  if (warp == 0 || warp == kTreeThreads / 32 - 1) {
    // ---------------- producers: whole warps on one path, one lane issues
    // (tma_load_3d_pair_warp). Warp 0 asks for keys (and Q's groups in front of a
    // run's), as far ahead as the ring has room; the last warp for the other
    // keys' values once Q.K^T is done (and for the rest of Q). With pages of 64
    // keys or more a group is one box [2 chunks][64 keys][64]; with smaller ones a
    // chunk is 64 / page boxes.
    const int half = warp == 0 ? rank : rank ^ 1;  // which 64 keys of a block this warp loads
    const int box_log = 6 - p.box_shift, boxes = 1 << box_log;
    const uint32_t box_bytes = 128u << p.box_shift;
    const int cache_rows = p.num_pages << p.page_shift, page_mask = (1 << p.page_shift) - 1;
    const uint32_t ring0 = smem_u32(smem + S::RING);
    const uint32_t kfull0 = bar(kTreeKFull), vfull0 = bar(kTreeVFull);
    const uint32_t issue = elect_lane(), arm = rank == 0 ? issue : 0u;  // the leader arms the shared barriers
    // Box `lane` of this warp's 64 keys of block j: whether the run has it, its
    // table entry (fetched a block ahead, and not looked at before row_of, so
    // that the warp does not wait for it), and its cache row; a box behind the
    // last position reads zeros from behind the cache.
    auto place = [&](int j) -> int64_t {
      return static_cast<int64_t>(j) * kTreeBlock + 64 * half + (static_cast<int64_t>(lane) << p.box_shift);
    };
    TreeRun sg = {};
    auto entry_of = [&](int j) -> int {
      int e = 0;
      if (lane < boxes && j < sg.j1 && place(j) < sg.len + sg.nodes)
        e = __ldg(p.table + static_cast<int64_t>(sg.b) * p.table_width + (place(j) >> p.page_shift));
      return e;
    };
    auto row_of = [&](int j, int entry) -> int {
      if (lane >= boxes || place(j) >= sg.len + sg.nodes) return cache_rows;
      if (entry < 0 || entry >= p.num_pages) {
        atomicCAS(p.err, 0, kErrPage);
        return cache_rows;
      }
      return (entry << p.page_shift) + static_cast<int>(place(j) & page_mask);
    };
    // Chunks 2 * pair_of and the next of the 64 keys whose rows the lanes hold, into group s.
    auto load_group = [&](uint32_t s, int pair_of, int rows, uint32_t barrier) {
      const uint32_t dst = ring0 + s * S::GROUP;
      if (box_log == 0) {
        tma_load_3d_pair_warp(dst, &tm_kv, barrier, 0, __shfl_sync(0xffffffffu, rows, 0), 2 * pair_of, issue);
      } else {
#pragma unroll 1
        for (int x = 0; x < boxes; ++x) {
          const int row = __shfl_sync(0xffffffffu, rows, x);
          tma_load_3d_pair_warp(dst + x * box_bytes, &tm_kv, barrier, 0, row, 2 * pair_of, issue);
          tma_load_3d_pair_warp(dst + S::CHUNK + x * box_bytes, &tm_kv, barrier, 0, row, 2 * pair_of + 1, issue);
        }
      }
    };
    bool ok = true;
    int g = 0, runs = 0;  // blocks and runs so far
    griddep_wait();       // q_abs; what comes before it here reads only what was there before that kernel began
    if (warp == 0) {
      const uint32_t rope0 = smem_u32(smem + S::ROPE), empty0 = bar(kTreeEmpty), rfull0 = bar(kTreeRopeFull);
      const uint32_t kfull0_leader = mapa_shared(kfull0, 0), rfull0_leader = mapa_shared(rfull0, 0);
      uint32_t ks = 0, parity = 0;  // the next group to fill
      if (busy) {
        work.b = start[0];
        work.tile = start[1];
        work.j = start[2];
        work.first = 1;
        tree_lengths(p, work.b, work.len, work.nodes);
        tree_extent(p, work.len, work.nodes, work.tiles, work.blocks);
      }
      while (ok && work.left > 0) {
        // This warp alone walks the share; the others take the run from here. The
        // slot is free: what the ring of groups does not hold any more is through,
        // and with seven groups a run or more, it holds parts of two.
        sg = work.next(p);
        if (lane == 0) {
          run_ring[runs & 3] = sg;
          mbar_arrive(bar(kTreeRun + (runs & 1)));
        }
        __syncwarp();
        int entry = entry_of(sg.j0);
        const int qrow = sg.b * p.N * p.H + sg.tile * kTreeRows + 64 * rank;
        const uint32_t landed = bar(kTreeQGroups + (runs++ & 1));
        mbar_arrive_expect_tx_warp(landed, S::Q_GROUPS * S::GROUP, issue);
#pragma unroll 1
        for (int i = 0; ok && i < S::Q_GROUPS; ++i) {
          if (!(ok = warp_wait_all(empty0 + 8 * ks, parity ^ 1, ab, kErrWaitConsumer))) break;
          mbar_arrive_expect_tx_warp(kfull0 + 8 * ks, 0, arm);  // keep step with the ring: nobody waits for these two
          mbar_arrive_expect_tx_warp(vfull0 + 8 * ks, 0, arm);
          tma_load_3d_pair_warp(ring0 + ks * S::GROUP, &tm_qabs, mapa_shared(landed, rank), 0, qrow, 2 * i, issue);
          if (++ks == S::GROUPS) ks = 0, parity ^= 1;
        }
        const int j1 = min(sg.j1, p.most_blocks);
#pragma unroll 1
        for (int j = sg.j0; ok && j < j1; ++j, ++g) {
          const int rows = row_of(j, entry);
          entry = entry_of(j + 1);
          // The rope slot: Q.K^T of the block two before has read it.
          if (g >= 2 && !(ok = warp_wait_all(bar(kTreeSFull + (g & 1)), ((g - 2) >> 1) & 1, ab, kErrWaitMma))) break;
          const uint32_t x = static_cast<uint32_t>(g) % S::ROPES;
          mbar_arrive_expect_tx_warp(rfull0 + 8 * x, 2 * S::CHUNK, arm);
#pragma unroll 1
          for (int i = 0; i < boxes; ++i)
            tma_load_2d_pair_warp(rope0 + x * S::CHUNK + i * box_bytes, &tm_pe, rfull0_leader + 8 * x, 0,
                                  __shfl_sync(0xffffffffu, rows, i), issue);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            if (!(ok = warp_wait_all(empty0 + 8 * ks, parity ^ 1, ab, kErrWaitConsumer))) break;
            mbar_arrive_expect_tx_warp(kfull0 + 8 * ks, 2 * S::GROUP, arm);
            load_group(ks, i, rows, kfull0_leader + 8 * ks);
            if (++ks == S::GROUPS) ks = 0, parity ^= 1;
          }
        }
        ok = ok && j1 == sg.j1;
      }
    } else {
      const uint32_t vfull0_leader = mapa_shared(vfull0, 0), qfull_leader = mapa_shared(bar(kTreeQFull), 0);
      const uint32_t q0 = smem_u32(smem + S::Q);
      uint32_t vs = 0;  // the next group to fill again
      int tails = 0;    // blocks with drafted keys so far
      bool more = busy;
      while (ok && more) {
        if (!(ok = warp_wait_all(bar(kTreeRun + (runs & 1)), (runs >> 1) & 1, ab, kErrWaitConsumer))) break;
        sg = run_ring[runs++ & 3];
        more = sg.flags & 2;
        int entry = entry_of(sg.j0);
        // Q's shared-memory part: Q.K^T of the run before is done. Rows past the
        // sequence's last belong to another sequence or to none, and are not stored.
        const int qrow = sg.b * p.N * p.H + sg.tile * kTreeRows + 64 * rank;
        mbar_arrive_expect_tx_warp(bar(kTreeQFull), 2 * S::Q_CHUNKS * S::CHUNK, arm);
        tma_load_3d_pair_warp(q0, &tm_qabs, qfull_leader, 0, qrow, S::Q_TMEM, issue);
        tma_load_2d_pair_warp(q0 + 2 * S::CHUNK, &tm_q, qfull_leader, 128, qrow, issue);
        vs = (vs + S::Q_GROUPS) % S::GROUPS;
#pragma unroll 1
        for (int j = sg.j0; j < sg.j1; ++j, ++g) {
          const int rows = row_of(j, entry);
          entry = entry_of(j + 1);
          if (!(ok = warp_wait_all(bar(kTreeSFull + (g & 1)), (g >> 1) & 1, ab, kErrWaitMma))) break;
          // Over the groups this CTA is done with. In a block with drafted keys
          // the bytes count on a barrier of this CTA, and "P is written" tells the
          // issuer that they have landed.
          const bool tail = static_cast<int64_t>(j + 1) * kTreeBlock > sg.len;
          const uint32_t landed = bar(kTreeTail + (tails & 1));
          if (tail) {
            mbar_arrive_expect_tx_warp(landed, 2 * S::GROUP, issue);
            ++tails;
          }
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            mbar_arrive_expect_tx_warp(vfull0 + 8 * vs, tail ? 0 : S::GROUP, arm);
            if ((i & 1) != rank)
              load_group(vs, 2 * (i >> 1) + rank, rows, tail ? mapa_shared(landed, rank) : vfull0_leader + 8 * vs);
            if (++vs == S::GROUPS) vs = 0;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------- UMMA issuer, the whole warp (see umma_ss_pair_x4; each
      // lane waits for itself, and only the issuing lane's outcome counts):
      // Q.K^T of block j + 1, then P.V of block j
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 256, 0, 1);
      const uint64_t dring = smem_desc_sw128(smem_u32(smem + S::RING), 16, 1024);
      const uint64_t dring_mn = smem_desc_sw128(smem_u32(smem + S::RING), S::CHUNK, 1024);
      const uint64_t drope = smem_desc_sw128(smem_u32(smem + S::ROPE), 16, 1024);
      const uint64_t dq = smem_desc_sw128(smem_u32(smem + S::Q), 16, 1024);
      const uint64_t dp = smem_desc_sw128(smem_u32(smem + S::P), 16, 1024);
      const uint32_t kfull0 = bar(kTreeKFull), vfull0 = bar(kTreeVFull), empty0 = bar(kTreeEmpty), issue = elect_lane();
      bool ok = true;
      int g = 0, seg = 0, commits = 0;
      uint32_t ks = 0, kparity = 0, vs = 0, vparity = 0;  // the next groups of keys and of values
      griddep_wait();                                     // no bounded wait begins before that
      auto qk = [&](int block) -> bool {
        constexpr int kChunk = S::CHUNK >> 4, kGroup = S::GROUP >> 4;
        const uint32_t ts = tmem + kTreeColS;
        if (block > 0 && !mbar_wait_short(bar(kTreeSFree), (block - 1) & 1, ab, kErrWaitSoftmax)) return false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i == 3) {  // the rope chunk before the group that lands last
            const uint32_t x = static_cast<uint32_t>(block) % S::ROPES;
            if (!mbar_wait_short(bar(kTreeRopeFull) + 8 * x, (block / S::ROPES) & 1, ab, kErrWaitTma)) return false;
            tc_fence_after();
            umma_ss_pair_x4<2, 2>(ts, dq + (8 - S::Q_TMEM) * kChunk, drope + x * kChunk, idesc_qk, 1u, issue);
          }
          if (!mbar_wait_short(kfull0 + 8 * ks, kparity, ab, kErrWaitTma)) return false;
          tc_fence_after();
          const uint64_t k = dring + ks * kGroup;
          if (2 * i < S::Q_TMEM) {
            umma_ts_pair_x4<2>(ts, tmem + kTreeColQ + 64 * i, k, idesc_qk, i > 0 ? 1u : 0u, issue);
            umma_ts_pair_x4<2>(ts, tmem + kTreeColQ + 64 * i + 32, k + kChunk, idesc_qk, 1u, issue);
          } else {
            const uint64_t a = dq + (2 * i - S::Q_TMEM) * kChunk;
            umma_ss_pair_x4<2, 2>(ts, a, k, idesc_qk, 1u, issue);
            umma_ss_pair_x4<2, 2>(ts, a + kChunk, k + kChunk, idesc_qk, 1u, issue);
          }
          if (++ks == S::GROUPS) ks = 0, kparity ^= 1;
        }
        umma_commit_pair_warp(bar(kTreeSFull + (block & 1)), 0x3, issue);
        ++commits;
        return true;
      };
      auto pv = [&](int block, bool fresh) -> bool {
        constexpr int kChunk = S::CHUNK >> 4, kGroup = S::GROUP >> 4;
        if (!mbar_wait_short(bar(kTreePFull), block & 1, ab, kErrWaitSoftmax)) return false;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // values [256 (i / 2), + 256) of keys [64 (i % 2), + 64)
          if (!mbar_wait_short(vfull0 + 8 * vs, vparity, ab, kErrWaitTma)) return false;
          tc_fence_after();
          umma_ss_pair_x4<2, 128>(tmem + 128u * (i >> 1), dp + (i & 1) * kChunk, dring_mn + vs * kGroup, idesc_pv,
                                  (!fresh || (i & 1)) ? 1u : 0u, issue);
          umma_commit_pair_warp(empty0 + 8 * vs, 0x3, issue);
          if (++vs == S::GROUPS) vs = 0, vparity ^= 1;
        }
        umma_commit_pair_warp(bar(kTreePVDone), 0x3, issue);
        ++commits;
        return true;
      };
      bool more = busy;
      while (ok && more) {
        if (!(ok = mbar_wait_short(bar(kTreeQFull), seg & 1, ab, kErrWaitTma))) break;
        if (!(ok = mbar_wait_short(bar(kTreeQReady), seg & 1, ab, kErrWaitSoftmax))) break;
        const int n = run_ring[seg & 3].j1 - run_ring[seg & 3].j0;
        more = run_ring[seg & 3].flags & 2;
        for (int i = 0; i < S::Q_GROUPS; ++i) {  // Q's groups are free: nothing else has read them
          umma_commit_pair_warp(empty0 + 8 * ks, 0x3, issue);
          if (++ks == S::GROUPS) ks = 0, kparity ^= 1;
          if (++vs == S::GROUPS) vs = 0, vparity ^= 1;
        }
        tc_fence_after();
#pragma unroll 1
        for (int j = -1; ok && j < n; ++j) {
          if (j + 1 < n) ok = qk(g + j + 1);
          if (ok && j >= 0) ok = pv(g + j, j == 0);
        }
        g += n;
        ++seg;
      }
      if (!ok && commits > 0) {
        umma_commit_pair_warp(bar(kTreeDrain), 0x1, issue);
        mbar_wait_drain(bar(kTreeDrain), 0);
      }
    }
  } else {
    // ---------------- softmax. Quadrant of tensor-memory lanes q, half ch of
    // its 64 key columns: row (32 q + lane) mod 64, keys 64 (q / 2) + 32 ch ..
    // + 32 of the block.
    const int quad = warp & 3, ch = (warp - 2) >> 2;
    const int row = (32 * quad + lane) & 63, lh = quad >> 1, part = 2 * lh + ch;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* xchg = reinterpret_cast<float*>(smem + S::XCHG);
    uint8_t* prow = smem + S::P + lh * S::CHUNK + row * 128;
    const float c = p.scale_log2;
    const uint32_t p_full = mapa_shared(bar(kTreePFull), 0), s_free = mapa_shared(bar(kTreeSFree), 0);
    bool ok = true;
    int g = 0, tails = 0, turn = 0, meets = 0, runs = 0;  // runs: whose Q has been loaded
    // The four threads' values of this row.
    auto exchange = [&](float v, float (&all)[4]) -> bool {
      float* x = xchg + (turn & 1) * 256;
      x[part * 64 + row] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kTreeXchg + (quad & 1)));
      if (!warp_wait_all(bar(kTreeXchg + (quad & 1)), turn & 1, ab, kErrWaitSoftmax)) return false;
      ++turn;
#pragma unroll
      for (int i = 0; i < 4; ++i) all[i] = x[i * 64 + row];
      return true;
    };
    // The eight warps meet.
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kTreeOut));
      return warp_wait_all(bar(kTreeOut), meets++ & 1, ab, kErrWaitSoftmax);
    };
    // Q's groups (positions `at` and on of the ring) into tensor memory: with M =
    // 128 both lane r and lane r + 64 hold row r; this warp's three chunks of
    // its lanes' rows.
    auto load_q = [&](int at) -> bool {
      if (!warp_wait_all(bar(kTreeQGroups + (runs & 1)), (runs >> 1) & 1, ab, kErrWaitTma)) return false;
      ++runs;
#pragma unroll 1
      for (int i = 0; i < 3; ++i) {
        const int c = 3 * ch + i;
        const uint8_t* src = smem + S::RING + (at + (c >> 1)) % S::GROUPS * S::GROUP + (c & 1) * S::CHUNK + row * 128;
        uint32_t v[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + ((k ^ (row & 7)) << 4));
          v[4 * k] = w.x, v[4 * k + 1] = w.y, v[4 * k + 2] = w.z, v[4 * k + 3] = w.w;
        }
        tmem_st32(tl + kTreeColQ + 32u * c, v);
      }
      fence_proxy_async_smem();  // the groups are filled again by TMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(bar(kTreeQReady), 0));
      return true;
    };
    griddep_wait();
    if (busy) ok = load_q(0);
    bool more = busy;
    while (ok && more) {
      const TreeRun sg = run_ring[(runs - 1) & 3];
      more = sg.flags & 2;
      const int r = sg.tile * kTreeRows + 64 * rank + row;  // row of the sequence: node * H + head
      const int live = sg.nodes * p.H;
      const bool has_tail = static_cast<int64_t>(sg.j1) * kTreeBlock > sg.len;
      const uint64_t sees = has_tail ? tree_ancestors(p, sg.b, min(r / p.H, kTreeMax)) : 0ull;
      const int total = sg.len + sg.nodes;
      float m_run = -INFINITY, l_run = 0.f;
#pragma unroll 1
      for (int j = sg.j0; j < sg.j1; ++j, ++g) {
        if (!(ok = warp_wait_all(bar(kTreeSFull + (g & 1)), (g >> 1) & 1, ab, kErrWaitMma))) break;
        tc_fence_after();
        float x[32];
        tmem_ld32(tl + kTreeColS + 32u * ch, *reinterpret_cast<uint32_t(*)[32]>(x));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(s_free);
        const int64_t t0 = static_cast<int64_t>(j) * kTreeBlock;
        const bool tail = t0 + kTreeBlock > sg.len;
        if (tail) {
          const uint32_t keep = tree_keep(t0 + 64 * lh + 32 * ch, sg.len, sees);
          uint32_t low = 0u;  // seen, with a score of -inf
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            low |= x[i] == -INFINITY ? 1u << i : 0u;
            x[i] = (keep >> i) & 1 ? x[i] : -INFINITY;
          }
          // Such a key's weight is 0, and 0 times a value that is not finite is NaN;
          // the values no longer say so (see below), so the sum does.
          if ((low & keep) != 0u &&
              tree_latent_not_finite(p.kv, p.table + static_cast<int64_t>(sg.b) * p.table_width, p.page_shift, p.num_pages,
                                     t0 + 64 * lh + 32 * ch, total, low & keep))
            l_run = NAN;
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(x[i], x[4 + i], x[8 + i]);
#pragma unroll
        for (int k0 = 12; k0 < 28; k0 += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], x[k0 + i], x[k0 + 4 + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[28 + i]);
        float all[4];
        if (!(ok = exchange(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), all))) break;
        // Lazy rescaling: the running maximum moves only when a block exceeds
        // it by more than 8 (in log2), so P < 2^8 and O is rarely touched.
        const float m_new = fmaxf(m_run, fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3])) * c);
        const bool resc = (m_new - m_run) > 8.f;
        float alpha = 1.f;
        if (resc) {
          alpha = ex2_approx(m_run - m_new);
          m_run = m_new;
        }
        const float nb = (m_run == -INFINITY) ? 0.f : -m_run;
        float sm[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          fma2_scalar(x[2 * i], x[2 * i + 1], c, nb);
          const float p0 = ex2_approx(x[2 * i]);
          const float p1 = ex2_approx(x[2 * i + 1]);
          add2(sm[2 * (i & 1)], sm[2 * (i & 1) + 1], p0, p1);
          pk[i] = pack_bf16x2(p0, p1);
        }
        l_run = l_run * alpha + ((sm[0] + sm[1]) + (sm[2] + sm[3]));
        // P.V of the block before must be done before P is overwritten and O rescaled.
        if (g > 0 && !(ok = warp_wait_all(bar(kTreePVDone), (g - 1) & 1, ab, kErrWaitMma))) break;
        if (j > sg.j0 && __any_sync(0xffffffffu, resc)) {
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(tl + 128u * ch + c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tl + 128u * ch + c0, o);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(prow + (((4 * ch + i) ^ (row & 7)) << 4)) =
              make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        if (tail) {
          // The values from the first drafted key on: those behind the last
          // position hold whatever the page held before, and 0 * NaN is
          // NaN, so they are zeroed; so is what is not finite in a drafted
          // key's values. A row that sees such a key gets its NaN from the score,
          // which then is not finite, or from its sum where the score is -inf.
          if (!(ok = warp_wait_all(bar(kTreeTail + (tails & 1)), (tails >> 1) & 1, ab, kErrWaitTma))) break;
          ++tails;
          {
            const int who = static_cast<int>(threadIdx.x) - 64;  // 256 threads: piece who % 32 of key who / 32
            const int piece = who & 31, h = piece >> 4, chunk = (piece >> 3) & 1;
            for (int k = static_cast<int>(max(int64_t(0), sg.len - t0)) + (who >> 5); k < kTreeBlock; k += 8) {
              uint4* at = reinterpret_cast<uint4*>(smem + S::RING + (S::Q_GROUPS * runs + 4 * g + 2 * h + (k >> 6)) % S::GROUPS * S::GROUP +
                                                   chunk * S::CHUNK + (k & 63) * 128 + (piece & 7) * 16);
              uint4 v = *at;
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (t0 + k >= total) {
                  w[i] = 0u;
                } else {
                  if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
                  if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0x0000ffffu;
                }
              }
              *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        // P (and the zeroed values) is in this SM's own shared memory, where its
        // tensor core reads it: each lane's fence has put its stores there before
        // lane 0 arrives (see mbar_arrive_remote for what that rests on). A
        // cluster-scope release here, which would order them for the other SM's
        // threads by the memory model, took 1300 to 2100 clk a block; by one idle
        // thread of the second CTA for its eight warps, 64 nodes over 32768 keys took
        // 638 us for 460, the batch over e4m3 weights 216 for 187.
        if (lane == 0) mbar_arrive_remote(p_full);
      }
      if (!ok) break;
      // ---------------- the run's result: o_lat, or its part of it. The next
      // run's Q first: its products have no more use for this one's.
      if (more && !(ok = load_q(4 * g + S::Q_GROUPS * runs))) break;
      float all[4];
      if (!(ok = exchange(l_run, all) && warp_wait_all(bar(kTreePVDone), (g - 1) & 1, ab, kErrWaitMma))) break;
      tc_fence_after();
      const float l = (all[0] + all[1]) + (all[2] + all[3]);
      const int v0 = 256 * ch + 128 * lh;  // this thread's 128 of the 512 values
      if (sg.j1 - sg.j0 == sg.blocks) {
        // Through P's shared memory, 32 of each thread's values at a time, so that
        // 64 consecutive bytes of a row leave together: stored by the threads
        // that hold them, 16 bytes a row, a tile took 8k clk.
        float inv = 1.f / l;  // l = 0: no finite score, 0 / 0
        if (p.v_scale != nullptr) inv *= __ldg(p.v_scale + (2 * (r % p.H) + 1) * 4 + (v0 >> 7));
        uint8_t* const stage = smem + S::P;
        const int who = static_cast<int>(threadIdx.x) - 64, piece = who & 15, r0 = sg.tile * kTreeRows + 64 * rank;
        // piece: 16 bytes of one of the four threads' 64 (values 128 (piece / 4) ...)
        uint8_t* const dst = reinterpret_cast<uint8_t*>(p.olat + (static_cast<int64_t>(sg.b) * p.N * p.H + r0) * 512) +
                             (piece >> 2) * 256 + (piece & 3) * 16;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tl + 128u * ch + c0, o);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stage + row * 256 + (((4 * (2 * ch + lh) + i) ^ (row & 7)) << 4)) =
                make_uint4(pack_bf16x2(__uint_as_float(o[8 * i + 0]) * inv, __uint_as_float(o[8 * i + 1]) * inv),
                           pack_bf16x2(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv),
                           pack_bf16x2(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv),
                           pack_bf16x2(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv));
          if (!(ok = meet())) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = (who >> 4) + 16 * i;
            if (r0 + rr < live)
              *reinterpret_cast<uint4*>(dst + rr * 1024 + c0 * 2) =
                  *reinterpret_cast<const uint4*>(stage + rr * 256 + ((piece ^ (rr & 7)) << 4));
          }
          if (!(ok = meet())) break;
        }
      } else {
        const int slot = 2 * pair + (sg.flags & 1 ? 0 : 1);
        const int tr = 64 * rank + row;
        float* dst = p.part_o + static_cast<int64_t>(slot) * kTreeSlotFloats + (v0 / 4 * kTreeRows + tr) * 4;
        if (part == 0) p.part_ml[slot * kTreeRows + tr] = make_float2(m_run, l);
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tl + 128u * ch + c0, o);
          if (r < live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(dst + (c0 / 4 + i) * kTreeRows * 4) =
                  make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                              __uint_as_float(o[4 * i + 3]));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // After a wait has run out in any warp, what others have asked for must land
  // before the CTA can exit.
  if (ab.raised()) spin_ns(2000000);
  cluster_sync();  // the leader's UMMAs read the other CTA's shared memory until here
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Joins the tiles that several pairs shared, and zeroes the rows of nodes that
// are not there. Thread: one row of a tile, VALUES of its values; with M the
// largest of the parts' maxima, o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p
// over the pairs p whose shares meet the tile, in their order. The pairs are
// found side by side, one per thread: one after the other, with their 64-bit
// divisions, took 40 us for a tile of eight parts. Three shapes, by the tiles:
//   many   16 values, two parts on their way, 16 blocks a tile
//   some   4 values, eight parts, 64 blocks: where many would give fewer than two
//          blocks per SM. 8 tiles of 8 parts: a step of 93 us, 101 with 16 values;
//          16 tiles 97 and 97; 98 tiles with 8 values 4 us slower than with 16
//   few    4 values, and four teams of a block that take every fourth part, 128
//          blocks: where all of them are resident at once. One tile of 74 parts
//          (one sequence of 32768, one token of 128 heads) 87 us, 99 as some, 148
//          as many; 2 tiles 84 and 90, 3 tiles 92 and 93, 6 tiles 102 and 100
template <int VALUES, int TEAMS>
struct TreeJoin {
  static constexpr int TEAM = TEAMS > 1 ? kTreeRows : 256;              // threads
  static constexpr int THREADS = TEAM * TEAMS;
  static constexpr int BLOCKS = kTreeRows * (512 / VALUES) / TEAM;      // per tile
  static constexpr int QUADS = VALUES / 4, BATCH = TEAMS > 1 ? 4 : 32 / VALUES;  // parts on their way at once
};
static_assert(kTreeMaxPairs <= 96, "three warps look for the parts");

template <int VALUES, int TEAMS>
__global__ void __launch_bounds__(TreeJoin<VALUES, TEAMS>::THREADS, TEAMS > 1 ? 2 : 1)
tree_combine_kernel(const TreeParams p, int pairs) {
  using J = TreeJoin<VALUES, TEAMS>;
  constexpr int QUADS = J::QUADS, BATCH = J::BATCH;
  __shared__ int slots[96];
  __shared__ int found[3];
  griddep_launch();
  griddep_wait();
  const int all_tiles = (p.N * p.H + kTreeRows - 1) / kTreeRows;
  const int at = static_cast<int>(blockIdx.x) / J::BLOCKS, b = at / all_tiles, tile = at % all_tiles;
  const int team = static_cast<int>(threadIdx.x) / J::TEAM;
  const int item = static_cast<int>(blockIdx.x) % J::BLOCKS * J::TEAM + static_cast<int>(threadIdx.x) % J::TEAM;
  const int tr = item & 127, v0 = (item >> 7) * VALUES;
  const int r = tile * kTreeRows + tr;
  // Asked for before the lengths are looked at.
  const int64_t units = p.ustart[p.B], extra = p.ustart[p.B + 1], first = p.ustart[b];
  int len, nodes, tiles, blocks;
  tree_lengths(p, b, len, nodes);
  tree_extent(p, len, nodes, tiles, blocks);
  // Part of pair c, if it has one, in the order of the pairs.
  const int c = static_cast<int>(threadIdx.x);
  int slot = -1;
  if (c < 96) {
    if (c < pairs && tile < tiles) {
      // Its share [s0, s1) as blocks of this tile, counted from the first.
      const int64_t lo = first + static_cast<int64_t>(tile) * (blocks + extra) + extra;
      int64_t s0, s1;
      tree_share(units, c, pairs, s0, s1);
      s0 -= lo, s1 -= lo;
      const int64_t j0 = max(s0, int64_t(0)), j1 = min(s1, int64_t(blocks));
      if (j0 < j1 && j1 - j0 < blocks) slot = 2 * c + (s0 >= -extra ? 0 : 1);
    }
    const uint32_t mine = __ballot_sync(0xffffffffu, slot >= 0);
    if ((c & 31) == 0) found[c >> 5] = static_cast<int>(mine);
  }
  __syncthreads();
  const int n0 = __popc(found[0]), n1 = __popc(found[1]), n = n0 + n1 + __popc(found[2]);
  if (slot >= 0)
    slots[(c >= 64 ? n0 + n1 : c >= 32 ? n0 : 0) + __popc(static_cast<uint32_t>(found[c >> 5]) & ((1u << (c & 31)) - 1))] = slot;
  __syncthreads();
  uint2* dst = reinterpret_cast<uint2*>(p.olat + (static_cast<int64_t>(b) * p.N * p.H + r) * 512 + v0);
  const bool live = r < nodes * p.H;
  if (!live && r < p.N * p.H && team == 0) {
#pragma unroll
    for (int k = 0; k < QUADS; ++k) dst[k] = make_uint2(0u, 0u);
  }
  if (n == 0) return;  // one pair's alone
  float M = -INFINITY;
#pragma unroll 8
  for (int i = team; live && i < n; i += TEAMS) M = fmaxf(M, p.part_ml[slots[i] * kTreeRows + tr].x);
  const float base = M == -INFINITY ? 0.f : M;
  float4 acc[QUADS];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < QUADS; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = team; live && i0 < n; i0 += BATCH * TEAMS) {
    float2 ml[BATCH];
    float4 v[BATCH][QUADS];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (i0 + u * TEAMS >= n) continue;
      const int s = slots[i0 + u * TEAMS];
      const float4* src = reinterpret_cast<const float4*>(p.part_o + static_cast<int64_t>(s) * kTreeSlotFloats) +
                          v0 / 4 * kTreeRows + tr;
      ml[u] = p.part_ml[s * kTreeRows + tr];
#pragma unroll
      for (int k = 0; k < QUADS; ++k) v[u][k] = src[k * kTreeRows];
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (i0 + u * TEAMS >= n) continue;
      const float w = ex2_approx(ml[u].x - base);  // 0 for a part of which the row sees no key, or none with a finite score
      sum = fmaf(w, ml[u].y, sum);
#pragma unroll
      for (int k = 0; k < QUADS; ++k)
        acc[k] = make_float4(fmaf(w, v[u][k].x, acc[k].x), fmaf(w, v[u][k].y, acc[k].y), fmaf(w, v[u][k].z, acc[k].z),
                             fmaf(w, v[u][k].w, acc[k].w));
    }
  }
  if constexpr (TEAMS > 1) {
    __shared__ float joined[TEAMS - 1][2 + VALUES][kTreeRows];
    if (team > 0) {
      float(*j)[kTreeRows] = joined[team - 1];
      j[0][tr] = M;
      j[1][tr] = sum;
#pragma unroll
      for (int k = 0; k < QUADS; ++k)
        j[4 * k + 2][tr] = acc[k].x, j[4 * k + 3][tr] = acc[k].y, j[4 * k + 4][tr] = acc[k].z, j[4 * k + 5][tr] = acc[k].w;
    }
    __syncthreads();
    if (team > 0) return;
    float top = M;
#pragma unroll
    for (int i = 0; i < TEAMS - 1; ++i) top = fmaxf(top, joined[i][0][tr]);
    const float all = top == -INFINITY ? 0.f : top, own = ex2_approx(M - all);
    sum *= own;
#pragma unroll
    for (int k = 0; k < QUADS; ++k) acc[k] = make_float4(acc[k].x * own, acc[k].y * own, acc[k].z * own, acc[k].w * own);
#pragma unroll
    for (int i = 0; i < TEAMS - 1; ++i) {
      const float(*j)[kTreeRows] = joined[i];
      const float w = ex2_approx(j[0][tr] - all);
      sum = fmaf(w, j[1][tr], sum);
#pragma unroll
      for (int k = 0; k < QUADS; ++k)
        acc[k] = make_float4(fmaf(w, j[4 * k + 2][tr], acc[k].x), fmaf(w, j[4 * k + 3][tr], acc[k].y),
                             fmaf(w, j[4 * k + 4][tr], acc[k].z), fmaf(w, j[4 * k + 5][tr], acc[k].w));
    }
  }
  if (!live) return;
  float inv = 1.f / sum;
  if (p.v_scale != nullptr) inv *= __ldg(p.v_scale + (2 * (r % p.H) + 1) * 4 + (v0 >> 7));
  uint32_t o[2 * QUADS];
#pragma unroll
  for (int k = 0; k < QUADS; ++k) {
    o[2 * k] = pack_bf16x2(acc[k].x * inv, acc[k].y * inv);
    o[2 * k + 1] = pack_bf16x2(acc[k].z * inv, acc[k].w * inv);
  }
  if constexpr (QUADS == 1) {
    *dst = make_uint2(o[0], o[1]);
  } else {
#pragma unroll
    for (int k = 0; k < QUADS / 2; ++k)
      reinterpret_cast<uint4*>(dst)[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
  }
}

}  // namespace mla
