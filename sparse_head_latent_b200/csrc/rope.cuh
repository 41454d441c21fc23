// rope.cuh -- rotary positions, alone and fused with the latent RMSNorm that
// fills the cache (sm_100a).
//
// Rotation of pair i of a head at position s:
//   (u, v) -> m (u cos a - v sin a, v cos a + u sin a),   a = s f_i,
// with f_i = base^(-2i/64), scaled for long contexts when the table is made
// (mla_rope_init). The table holds f_i / 2 pi (turns per position) as a 64-bit
// binary fraction, right to two units, so that s f_i mod one turn is one integer
// product with an error of s 2^-63 turns, 2^-32 at the farthest position: the
// angle of a position in the millions is as exact as that of the first (a 32-bit
// float product is off by s 2^-25 radians, 0.03 at a million). The leading 32 bits
// of the fraction then become a float: of half a turn, 2^-31 from the table, 2^-31
// from the bits left out and 2^-25 from the rounding are below 2^-24 together.
//
// Both kernels read and write every byte once and do a few operations per
// byte, so memory bounds them; at one token it is the launch.
#pragma once

#include "ptx.cuh"

namespace mla {

constexpr int kRopeDim = 64;
constexpr int kRopePairs = kRopeDim / 2;

struct RopeTable {
  uint64_t turns[kRopePairs];  // f_i / 2 pi in units of 2^-64 turns
  float magnitude;             // multiplies cos and sin
  int layout;                  // MLA_ROPE_INTERLEAVED or MLA_ROPE_HALF
};

// The table's frequencies by a generic address: as a constant each lane's own
// index would be read one after the other.
__device__ __forceinline__ const uint64_t* rope_turns(const RopeTable& tab) {
  const uint64_t* t = tab.turns;
  asm("" : "+l"(t));
  return t;
}

// m cos and m sin of position * f, the sine negated for the inverse.
__device__ __forceinline__ float2 rope_cos_sin(int position, uint64_t turns, float magnitude, bool inverse) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * magnitude, (inverse ? -s : s) * magnitude);
}

// One rotated pair, from and to bf16, rounded once.
__device__ __forceinline__ void rope_turn(float u, float v, float2 cs, float& a, float& b) {
  a = u * cs.x - v * cs.y;
  b = v * cs.x + u * cs.y;
}

__device__ __forceinline__ float2 bf16x2_float2(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

struct RopeParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t x_row, x_head, o_row, o_head;  // strides in elements
  int rows, heads;
  int chunks;        // 16-byte pieces of a head that are touched: all of it, or in place the rotary 8
  int first;         // the first of them within the head
  int rope_chunk;    // the piece where the rotary part starts
  int rows_per_block, head_blocks, heads_per_block;
  bool inverse;
  const int32_t* positions;
};

constexpr int kRopeThreads = 256;

// A group of `chunks` threads takes one head at a time, a thread the same
// 16-byte piece of each: pieces outside the rotary part are copied, a piece
// inside it is rotated with four cosines and sines that the thread computes
// once for its row and uses for all its heads. With many heads a block covers
// heads_per_block heads of one row, with few it covers several rows. Four
// heads are loaded before the first is stored, to keep loads in flight. 4096
// rows of 128 heads of 192, 403 MB: 62.5 us, 6.4 TB/s; in place, 128 of each head's
// 384 bytes, 134 MB read and written: 24.9 us, 5.4 TB/s; one row of 64 heads: 2 us.
template <bool HALF>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeTable tab, const RopeParams p) {
  const int groups = kRopeThreads / p.chunks;
  const int g = static_cast<int>(threadIdx.x) / p.chunks, piece = p.first + static_cast<int>(threadIdx.x) % p.chunks;
  if (g >= groups) return;
  int64_t row;
  int h, h_end, h_step;
  if (p.rows_per_block > 1) {
    if (g >= p.rows_per_block * p.heads) return;
    row = static_cast<int64_t>(blockIdx.x) * p.rows_per_block + g / p.heads;
    h = g % p.heads;
    h_end = h + 1;
    h_step = 1;
  } else {
    row = blockIdx.x / p.head_blocks;
    const int h0 = static_cast<int>(blockIdx.x % p.head_blocks) * p.heads_per_block;
    h = h0 + g;
    h_end = min(p.heads, h0 + p.heads_per_block);
    h_step = groups;
  }
  if (row >= p.rows) return;
  const int k = piece - p.rope_chunk;  // which of the 8 rotary pieces
  const bool turn = k >= 0 && k < 8;
  // HALF: the thread of rotary piece k turns pairs 4k .. 4k+3, whose two
  // halves are 8 bytes each at elements 4k and 32 + 4k of the rotary part.
  const int lo = HALF && turn ? p.rope_chunk * 8 + 4 * k : piece * 8;
  const __nv_bfloat16* x = p.x + row * p.x_row + lo;
  __nv_bfloat16* out = p.out + row * p.o_row + lo;
  uint4 w[4];
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h + i * h_step >= h_end) break;
      const __nv_bfloat16* s = x + (h + i * h_step) * p.x_head;
      if (HALF && turn) {
        const uint2 a = *reinterpret_cast<const uint2*>(s), b = *reinterpret_cast<const uint2*>(s + 32);
        w[i] = make_uint4(a.x, a.y, b.x, b.y);
      } else {
        w[i] = *reinterpret_cast<const uint4*>(s);
      }
    }
  };
  load();  // in flight while the cosines are made
  float2 cs[4];
  uint64_t turns[4];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turns[i] = rope_turns(tab)[4 * k + i];
  }
  if (turn) {
    const int pos = __ldg(p.positions + row);
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = rope_cos_sin(pos, turns[i], tab.magnitude, p.inverse);
  }
  while (h < h_end) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h + i * h_step >= h_end) break;
      __nv_bfloat16* d = out + (h + i * h_step) * p.o_head;
      if (!turn) {
        *reinterpret_cast<uint4*>(d) = w[i];
      } else if (HALF) {
        const float2 u0 = bf16x2_float2(w[i].x), u1 = bf16x2_float2(w[i].y);
        const float2 v0 = bf16x2_float2(w[i].z), v1 = bf16x2_float2(w[i].w);
        float a[4], b[4];
        rope_turn(u0.x, v0.x, cs[0], a[0], b[0]);
        rope_turn(u0.y, v0.y, cs[1], a[1], b[1]);
        rope_turn(u1.x, v1.x, cs[2], a[2], b[2]);
        rope_turn(u1.y, v1.y, cs[3], a[3], b[3]);
        *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
        *reinterpret_cast<uint2*>(d + 32) = make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
      } else {
        const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 uv = bf16x2_float2(in[e]);
          float a, b;
          rope_turn(uv.x, uv.y, cs[e], a, b);
          o[e] = pack_bf16x2(a, b);
        }
        *reinterpret_cast<uint4*>(d) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    h += 4 * h_step;
    if (h < h_end) load();
  }
}

struct AppendParams {
  const __nv_bfloat16* kv_a;  // [rows][576], row pitch kv_row
  int64_t kv_row;
  const void* weight;         // [512], fp32 or bf16
  bool weight_f32;
  float eps;
  const int32_t* positions;
  const int32_t* slots;       // cache row of each token, nullptr: row r
  __nv_bfloat16* kv;          // [cache_rows][512]
  __nv_bfloat16* pe;          // [cache_rows][64]
  int rows;
  int64_t cache_rows;
};

// One warp per token: c = w x / sqrt(mean x^2 + eps) over the 512 latent
// values (16 a lane, the sum in fp32 by shuffles) and the rotated key (one
// pair a lane), each rounded once, into the token's cache row. A token whose
// slot lies outside the cache is skipped. 16384 tokens, 38 MB: 9.9 us; 65536:
// 32 us, 4.7 TB/s. Four tokens a warp, all loaded first, took 13.4 us, a warp that
// loads its next token while it works on one 11.5: at 48 registers ten blocks
// share an SM, and that hides more.
template <bool HALF>
__global__ void __launch_bounds__(128)
cache_append_kernel(const __grid_constant__ RopeTable tab, const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  // Everything is loaded before anything is looked at.
  const uint64_t turns = rope_turns(tab)[lane];
  const int64_t slot = p.slots ? __ldg(p.slots + row) : row;
  const int pos = __ldg(p.positions + row);
  const __nv_bfloat16* src = p.kv_a + row * p.kv_row;
  uint4 w[2], gw[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(src) + lane + 32 * i);
  const __nv_bfloat16* key = src + 512 + (HALF ? lane : 2 * lane);
  const __nv_bfloat16 ku = key[0], kv = key[HALF ? 32 : 1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (p.weight_f32) {
      const uint4* wf = static_cast<const uint4*>(p.weight) + 2 * (lane + 32 * i);
      gw[2 * i] = __ldg(wf);
      gw[2 * i + 1] = __ldg(wf + 1);
    } else {
      gw[2 * i] = __ldg(static_cast<const uint4*>(p.weight) + lane + 32 * i);
    }
  }
  if (slot < 0 || slot >= p.cache_rows) return;
  const float u = __bfloat162float(ku), v = __bfloat162float(kv);
  float x[16];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = bf16x2_float2(in[e]);
      x[8 * i + 2 * e] = f.x;
      x[8 * i + 2 * e + 1] = f.y;
      sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = rsqrtf(sum * (1.f / 512.f) + p.eps);
  uint4* dst = reinterpret_cast<uint4*>(p.kv + slot * 512);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float g[8];
    if (p.weight_f32) {
      const uint32_t in[8] = {gw[2 * i].x,     gw[2 * i].y,     gw[2 * i].z,     gw[2 * i].w,
                              gw[2 * i + 1].x, gw[2 * i + 1].y, gw[2 * i + 1].z, gw[2 * i + 1].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = __uint_as_float(in[e]);
    } else {
      const uint32_t in[4] = {gw[2 * i].x, gw[2 * i].y, gw[2 * i].z, gw[2 * i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_float2(in[e]);
        g[2 * e] = f.x;
        g[2 * e + 1] = f.y;
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = pack_bf16x2(x[8 * i + 2 * e] * r * g[2 * e], x[8 * i + 2 * e + 1] * r * g[2 * e + 1]);
    dst[lane + 32 * i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  float a, b;
  rope_turn(u, v, rope_cos_sin(pos, turns, tab.magnitude, false), a, b);
  __nv_bfloat16* kd = p.pe + slot * 64;
  if (HALF) {
    kd[lane] = __float2bfloat16_rn(a);
    kd[32 + lane] = __float2bfloat16_rn(b);
  } else {
    reinterpret_cast<uint32_t*>(kd)[lane] = pack_bf16x2(a, b);
  }
}

}  // namespace mla
