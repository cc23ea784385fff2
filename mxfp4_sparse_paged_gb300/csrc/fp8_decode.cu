// fp8_paged_decode, fp8_block_decode: attention of the decode tokens over the 8-bit K/V cache, all
// pages of a sequence or the blocks (pages) that each token lists.
//
//   l_i = scale q . K_i,  out = sum_i softmax(l)_i V_i,  lse = ln sum_i exp(l_i)
//
// over the visible tokens i, K_i = 2^Ek code, V_i = 2^Ev code with one E for 32 tokens and a head.
//
// Bound: HBM, 256 bytes a cached token and KV head, while a tile has up to about 40 rows (query
// heads of one KV head, for all decode tokens of the sequence); the tensor pipe above.
//
// Work.  A tile is 16 M rows of one KV head of one owner (a sequence; with block lists a token),
// a unit 32 cached tokens of it.  All units of all tiles form one list, cut into equal ranges, one
// a CTA, and those into one for each group of M warps.  A group streams its units through a ring of
// shared-memory stages by tensor copies (TMA, 128-byte swizzle); warps of different groups never
// wait for one another before the end.  So the ragged lengths of a batch balance to within a unit.
//
// A unit in a warp (16 rows, everything in registers between the two products):
//   S = q K^T on mma m16n8k16: E4M3 codes widen to f16 exactly, q (bf16, scaled by a power of two)
//     too, so products are exact and sums fp32.  The k index of the fragments is a permutation of
//     the head's dims that lets a lane read 32 consecutive bytes of a key; with the swizzle no two
//     lanes of a quarter-warp meet in a bank.
//   p = 2^(S f - m + 8), f = scale log2(e) 2^Ek.  m moves only where a row's largest logit lies
//     2^7 above it, so a unit costs one vote and no reduction.  z sums p in fp32; P is f16 (11
//     bits: 2^-12 of a weight; weights down to 2^-22 of the largest keep all of them).
//   O += 2^Ev (P V): the accumulator fragment of S is the operand of the second product; a pair of
//     tokens' bytes is put side by side by byte permutes and widened to f16x2, exact.  The product
//     of 32 tokens is scaled in fp32, so scales of any two blocks may be any powers apart.
// The tensor memory path (tcgen05) has no use here at 16 rows: it computes 128-row tiles from shared
// memory, and would put scores and weights through tensor and shared memory on the way.
//
// Units where some row does not see all 32 tokens (a sequence's end) take a second form of the step:
// scores are masked, values that no row sees are zeroed (rows past the length may hold anything), and
// NaN codes that only some rows see reach those rows alone, by counting them in one more product.
//
// Ranges cut tiles.  A group keeps the tile it ends in until all groups of the CTA are done; then
// pieces of the same tile are joined in shared memory.  Pieces of a tile in several CTAs go to the
// workspace and are joined by a second kernel, in the order of the list: results repeat bit for bit.
#include <algorithm>
#include <cfloat>

#include <cuda.h>
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled

#include "fp8_kv.cuh"

namespace mx4 {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 24;                      // of all groups of a CTA
constexpr int kStepBytes = 2 * kSub * kFp8Row;   // K rows, V rows of a unit
constexpr int kMaxOwners = 2048;                 // sequences of a launch (their prefix sums)
constexpr int kRecRow = kHeadDim + 4;            // floats of a row in shared memory: O, m, z
constexpr float kUp = 8.f;                       // weights are 2^kUp at the reference
constexpr int64_t kMinUnits = 8;                 // of a CTA: one for each group of one warp

constexpr int kBarOff = kStages * kStepBytes;
constexpr int kSumOff = kBarOff + 2 * kStages * 8;
constexpr int kSegOff = kSumOff + kWarps * 8;    // [group]: last tile, the end of its units, first tile
constexpr int kPrefOff = kSegOff + kWarps * 24;
constexpr int kSmemBytes = kPrefOff + kMaxOwners * 8 + 1024;  // 1024: the stages' alignment

struct DecodeArgs {
  CUtensorMap kmap, vmap;
  const uint16_t* q;        // bf16 [T, H, 128]
  const uint8_t* ks;        // e8m0 [P, Hkv, 4]
  const uint8_t* vs;
  const int32_t* table;     // [B, W]
  int64_t W;
  const int32_t* seq_lens;  // [B]
  const int32_t* idx;       // [T, kb] (block lists) or null
  int kb;
  int64_t num_pages;
  int B, Q, H, Hkv, G;
  int R, RT;                // rows of an owner and KV head, tiles they take
  float scale;
  uint16_t* out;
  float* lse;
  float* rec;               // pieces: [CTA][0: of a tile begun before, 1: begun here][16 M][128], m z
  float* scratch;           // [CTA][8 warps][16][128], m z: tiles that a group ended but did not begin
  int64_t* meta;            // [CTA][3]: the tile that begins here and ends in a later CTA (-1: none), that CTA
  uint32_t* status;
};

// The list of units: how many a CTA takes, and where a group's range lies.
struct Cut {
  int64_t U, per;
  __device__ __forceinline__ int64_t lo(int64_t cta) const { return min(U, cta * per); }
  __device__ __forceinline__ int64_t group_lo(int64_t cta, int gi, int n) const {
    const int64_t a = lo(cta);
    return a + (lo(cta + 1) - a) * gi / n;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D = A B + C, not volatile: the compiler may order products by their operands.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}

__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int row, int head,
                                            int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// A warp's part of a tile: 16 rows, lane (g, c) = (lane / 4, lane % 4) holds rows g and g + 8,
// dims 32 c .. 32 c + 31 of O (o[j]: dims 32 c + j and 32 c + 16 + j of row g, then of row g + 8).
struct Rows {
  uint32_t qa[8][4];
  float o[16][4];
  float m[2], nb[2], z[2], f[2];  // reference, 8 - reference, sum, logit factor without 2^Ek
  int lim[2];                     // last visible token of rows g, g + 8
  int min_lim, max_lim;           // over the warp's rows

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = -INFINITY;
      nb[h] = 0.f;
      z[h] = 0.f;
    }
  }

  // q rows -> f16 fragments, scaled so that a row's largest element lies in [2^14, 2^15) (exact, but
  // for elements 2^-29 of it; rows whose largest is below 2^-86 lose bits).
  __device__ __forceinline__ void load_q(const uint16_t* p, bool real, int h, float scale, int lane) {
    const int c = lane & 3;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = real ? *reinterpret_cast<const uint4*>(p + 32 * c + 8 * i) : make_uint4(0, 0, 0, 0);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      am = max(am, max((w[i] << 17) >> 1, w[i] & 0x7FFF0000u));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    const int sigma = am == 0u ? 0 : min(100, max(-113, 14 - ((int)(am >> 23) - 127)));
    const float up = __uint_as_float((uint32_t)(127 + sigma) << 23) * (scale < 0.f ? -1.f : 1.f);
    f[h] = fabsf(scale) * 1.44269504f * __uint_as_float((uint32_t)(127 - sigma) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      qa[j][h] = half2_bits(bf16_bits_to_float(w[2 * j] & 0xFFFFu) * up,
                            bf16_bits_to_float(w[2 * j] >> 16) * up);
      qa[j][h + 2] = half2_bits(bf16_bits_to_float(w[2 * j + 1] & 0xFFFFu) * up,
                                bf16_bits_to_float(w[2 * j + 1] >> 16) * up);
    }
  }

  // One unit: 32 tokens from position tb on, K rows at ka and V rows at va (shared memory), Ek and
  // Ev as powers of two.  Tail: some row does not see all of them.
  template <bool Tail>
  __device__ __forceinline__ void step(uint32_t ka, uint32_t va, float ek, float ev, int tb, int lane) {
    const int g = lane >> 2, c = lane & 3;
    float s[4][4];
    {
      uint4 x[4][2];
      const uint32_t at = ka + g * kFp8Row;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        x[n][0] = lds128(at + n * 8 * kFp8Row + (((2 * c) ^ g) << 4));
        x[n][1] = lds128(at + n * 8 * kFp8Row + (((2 * c + 1) ^ g) << 4));
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint4 y = x[n][j >> 2];
          const uint32_t w = (j & 3) == 0 ? y.x : (j & 3) == 1 ? y.y : (j & 3) == 2 ? y.z : y.w;
          uint32_t b0, b1;
          e4m3x4_f16x2(w, b0, b1);
          mma(s[n], qa[j], b0, b1);
        }
    }
    const int rel0 = lim[0] - tb, rel1 = lim[1] - tb;  // last visible token of the unit
    if (Tail) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (8 * n + 2 * c + e > rel0) s[n][e] = -INFINITY;
          if (8 * n + 2 * c + e > rel1) s[n][2 + e] = -INFINITY;
        }
    }
    // factors stay finite (a score of 0 is a logit of 0 whatever the scales) or NaN
    float f0 = f[0] * ek, f1 = f[1] * ek;
    f0 = f0 > FLT_MAX ? FLT_MAX : f0;
    f1 = f1 > FLT_MAX ? FLT_MAX : f1;
    float mx0 = s[0][0], mx1 = s[0][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      mx0 = fmaxf(mx0, fmaxf(s[n][0], s[n][1]));
      mx1 = fmaxf(mx1, fmaxf(s[n][2], s[n][3]));
    }
    mx0 *= f0;
    mx1 *= f1;
    if (__any_sync(0xFFFFFFFFu, mx0 > m[0] + 7.f || mx1 > m[1] + 7.f)) {
      float t[2] = {mx0, mx1};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        t[h] = fmaxf(t[h], __shfl_xor_sync(0xFFFFFFFFu, t[h], 1));
        t[h] = fmaxf(t[h], __shfl_xor_sync(0xFFFFFFFFu, t[h], 2));
        if (t[h] > m[h] + 7.f) {
          const float down = ex2(m[h] - t[h]);
          m[h] = t[h];
          nb[h] = kUp - t[h];
          z[h] *= down;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j][2 * h] *= down;
            o[j][2 * h + 1] *= down;
          }
        }
      }
    }
    uint32_t pa[2][4];
    {
      float p[4][4], z0 = 0.f, z1 = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[n][e] = ex2(fmaf(s[n][e], f0, nb[0]));
          p[n][2 + e] = ex2(fmaf(s[n][2 + e], f1, nb[1]));
          if (Tail) {  // -inf times a factor of 0 or NaN is not -inf
            if (8 * n + 2 * c + e > rel0) p[n][e] = 0.f;
            if (8 * n + 2 * c + e > rel1) p[n][2 + e] = 0.f;
          }
        }
        z0 += p[n][0] + p[n][1];
        z1 += p[n][2] + p[n][3];
      }
      z[0] += z0;
      z[1] += z1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        pa[k][0] = half2_bits(p[2 * k][0], p[2 * k][1]);
        pa[k][1] = half2_bits(p[2 * k][2], p[2 * k][3]);
        pa[k][2] = half2_bits(p[2 * k + 1][0], p[2 * k + 1][1]);
        pa[k][3] = half2_bits(p[2 * k + 1][2], p[2 * k + 1][3]);
      }
    }
    uint4 y[2][4];  // tokens 16 k + 2 c + {0, 1, 8, 9}, dims 16 g .. 16 g + 15
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * k + 2 * c + (i & 1) + 8 * (i >> 1);
        y[k][i] = lds128(va + r * kFp8Row + ((g ^ (2 * c + (i & 1))) << 4));
        if (Tail && tb + r > max_lim) y[k][i] = make_uint4(0, 0, 0, 0);
      }
    uint32_t seen[2][4];
    float ev0 = ev, ev1 = ev;
    if (Tail) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * k + 2 * c + 8 * (i >> 1), rel = (i & 1) ? rel1 : rel0;
          seen[k][i] = (r <= rel ? 0x3C00u : 0u) | (r + 1 <= rel ? 0x3C000000u : 0u);
        }
      if (rel0 < 0) ev0 = 0.f;  // a scale of NaN reaches only rows that see its tokens
      if (rel1 < 0) ev1 = 0.f;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t b[2][4][2];  // [k][dim of the word][token pair]
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 ya = y[k][2 * h], yb = y[k][2 * h + 1];
          const uint32_t wa = w == 0 ? ya.x : w == 1 ? ya.y : w == 2 ? ya.z : ya.w;
          const uint32_t wb = w == 0 ? yb.x : w == 1 ? yb.y : w == 2 ? yb.z : yb.w;
          e4m3x4_f16x2(__byte_perm(wa, wb, 0x5140), b[k][0][h], b[k][1][h]);
          e4m3x4_f16x2(__byte_perm(wa, wb, 0x7362), b[k][2][h], b[k][3][h]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float t[4];
        if (Tail) {
          float nan[4];
          uint32_t ind[2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const __half2 v = *reinterpret_cast<const __half2*>(&b[k][i][h]);
              const __half2 n = __hisnan2(v);
              ind[k][h] = *reinterpret_cast<const uint32_t*>(&n);
              b[k][i][h] &= ~(((ind[k][h] >> 10) & 0x00010001u) * 0xFFFFu);
            }
          mma0(nan, seen[0], ind[0][0], ind[0][1]);
          mma(nan, seen[1], ind[1][0], ind[1][1]);
          mma0(t, pa[0], b[0][i][0], b[0][i][1]);
          mma(t, pa[1], b[1][i][0], b[1][i][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (nan[e] > 0.f) t[e] = __uint_as_float(0x7FC00000u);
        } else {
          mma0(t, pa[0], b[0][i][0], b[0][i][1]);
          mma(t, pa[1], b[1][i][0], b[1][i][1]);
        }
        float(&d)[4] = o[4 * w + i];
        d[0] = fmaf(ev0, t[0], d[0]);
        d[1] = fmaf(ev0, t[1], d[1]);
        d[2] = fmaf(ev1, t[2], d[2]);
        d[3] = fmaf(ev1, t[3], d[3]);
      }
    }
  }

  // z over the lanes of a row; O, m and z of row g + 8 h at p (128 floats), mz.
  __device__ __forceinline__ void sum_z() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      z[h] += __shfl_xor_sync(0xFFFFFFFFu, z[h], 1);
      z[h] += __shfl_xor_sync(0xFFFFFFFFu, z[h], 2);
    }
  }
  __device__ __forceinline__ void put(int h, float* p, float* mz, int lane) const {
    const int c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(p + 32 * c + 16 * e + 4 * i) =
            make_float4(o[4 * i][2 * h + e], o[4 * i + 1][2 * h + e], o[4 * i + 2][2 * h + e],
                        o[4 * i + 3][2 * h + e]);
    if (c == 0) {
      mz[0] = m[h];
      mz[1] = z[h];
    }
  }
};

// A finished row's value and lse from O (units 2^(m - kUp)), m and z.
__device__ __forceinline__ float row_lse(float m, float z) {
  return z == 0.f ? -INFINITY : (m - kUp + log2f(z)) * 0.69314718f;
}

struct Tile {
  int owner, head, rt;
};
__device__ __forceinline__ Tile tile_of(const DecodeArgs& a, int64_t tile) {
  const int per = a.Hkv * a.RT;
  Tile t;
  t.owner = (int)(tile / per);
  const int r = (int)(tile - (int64_t)t.owner * per);
  t.head = r / a.RT;
  t.rt = r - t.head * a.RT;
  return t;
}

// Row r of a tile's owner: the decode token and query head it is.
template <bool Lists>
__device__ __forceinline__ int64_t row_of(const DecodeArgs& a, const Tile& t, int r) {
  const int j = Lists ? 0 : r / a.G;
  const int64_t tok = Lists ? t.owner : (int64_t)t.owner * a.Q + j;
  return tok * a.H + t.head * a.G + (r - j * a.G);
}

// A piece of a row onto a sum with the reference ref.
__device__ __forceinline__ void add_piece(float4& acc, float& z, float4 v, float pm, float pz, float ref) {
  // (a piece without a reference holds nothing, or NaN)
  const float f = pm == -INFINITY ? (pz == 0.f ? 0.f : 1.f) : ex2(pm - ref);
  z = fmaf(f, pz, z);
  acc.x = fmaf(f, v.x, acc.x);
  acc.y = fmaf(f, v.y, acc.y);
  acc.z = fmaf(f, v.z, acc.z);
  acc.w = fmaf(f, v.w, acc.w);
}
template <bool Lists>
__device__ __forceinline__ void put_row(const DecodeArgs& a, const Tile& t, int row, float4 acc, float m,
                                        float z, int lane) {
  const float inv = z == 0.f ? 0.f : 1.f / z;
  const int64_t at = row_of<Lists>(a, t, row);
  *reinterpret_cast<uint2*>(a.out + at * kHeadDim + 4 * lane) =
      make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[at] = row_lse(m, z);
}

// ---------------------------------------------------------------------------

template <int M, bool Lists>
__global__ void __launch_bounds__(kThreads, 1) fp8_decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int NG = kWarps / M, S = kStages / NG;  // groups, stages of a group
  static_assert(S <= 32, "a unit is looked up at most 32 ahead");
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = warp / M, wig = warp % M;
  uint64_t* const full = reinterpret_cast<uint64_t*>(sm + kBarOff) + group * S;
  uint64_t* const empty = full + kStages;
  int64_t* const sums = reinterpret_cast<int64_t*>(sm + kSumOff);
  int64_t* const seg = reinterpret_cast<int64_t*>(sm + kSegOff);
  int64_t* const pref = reinterpret_cast<int64_t*>(sm + kPrefOff);
  if (tid < kStages) {
    mbar_init(smem_addr(reinterpret_cast<uint64_t*>(sm + kBarOff) + tid), 1);
    mbar_init(smem_addr(reinterpret_cast<uint64_t*>(sm + kBarOff) + kStages + tid), M);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- units of the owners before each one
  const int HR = a.Hkv * a.RT;
  auto seq_units = [&](int s) {
    const int L = a.seq_lens[s];
    const bool ok = L >= 0 && L <= a.W * kPageTokens;
    if (!ok && blockIdx.x == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    return ok ? (L + kSub - 1) / kSub : 0;
  };
  Cut cut;
  if (Lists) {
    if (blockIdx.x == 0)
      for (int s = tid; s < a.B; s += kThreads) seq_units(s);
    cut.U = (int64_t)a.B * a.Q * HR * a.kb * kPageSubs;
    __syncthreads();
  } else {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int s0 = min(a.B, tid * per), s1 = min(a.B, s0 + per);
    int64_t sum = 0;
    for (int s = s0; s < s1; ++s) sum += seq_units(s);
    int64_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
    for (int w = 0; w < warp; ++w) before += sums[w];
    for (int s = s0; s < s1; ++s) {
      before += seq_units(s);
      pref[s] = before;
    }
    __syncthreads();
    cut.U = pref[a.B - 1] * HR;
  }
  cut.per = max((cut.U + gridDim.x - 1) / gridDim.x, (int64_t)kMinUnits);

  // ---- owners without units: their rows are empty
  for (int64_t t = blockIdx.x; !Lists && t < (int64_t)a.B * a.Q; t += gridDim.x) {
    const int s = (int)(t / a.Q);
    if (pref[s] != (s ? pref[s - 1] : 0)) continue;
    for (int i = tid; i < a.H * kHeadDim / 8; i += kThreads)
      reinterpret_cast<uint4*>(a.out + t * a.H * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.H; i += kThreads) a.lse[t * a.H + i] = -INFINITY;
  }

  const int64_t u0 = cut.group_lo(blockIdx.x, group, NG);
  const int64_t n64 = cut.group_lo(blockIdx.x, group + 1, NG) - u0;

  // ---- what unit u is: its tile, first token, page (-1: skipped) and scales
  struct Unit {
    int tile, tb, page, sc;
    int i, n;  // number in its tile, units of the tile
  };
  auto resolve = [&](int64_t k) {
    Unit r{0, 0, -1, 0, 0, 1};
    if (k >= n64) return r;
    const int64_t u = u0 + k;
    int owner, head;
    if (Lists) {
      r.n = a.kb * kPageSubs;
      const int64_t tile = u / r.n;
      r.i = (int)(u - tile * r.n);
      r.tile = (int)tile;
      const Tile t = tile_of(a, tile);
      owner = t.owner / a.Q;
      head = t.head;
      const int b = a.idx[(int64_t)t.owner * a.kb + r.i / kPageSubs];
      if (b < 0) return r;
      const int64_t L = a.seq_lens[owner];
      const int64_t p = L - a.Q + t.owner % a.Q;
      if (L < 0 || L > a.W * kPageTokens) return r;
      if (p < 0 || b > p / kPageTokens) {
        flag(a.status, MX4_STATUS_BAD_INDEX);
        return r;
      }
      r.tb = b * kPageTokens + (r.i % kPageSubs) * kSub;
      if (r.tb > p) return r;
    } else {
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (pref[mid] * HR > u) hi = mid; else lo = mid + 1;
      }
      owner = lo;
      const int64_t before = lo ? pref[lo - 1] : 0;
      r.n = (int)(pref[lo] - before);
      const int64_t v = u - before * HR;
      const int in = (int)(v / r.n);
      r.i = (int)(v - (int64_t)in * r.n);
      r.tile = lo * HR + in;
      head = in / a.RT;
      r.tb = r.i * kSub;
    }
    const int32_t page = a.table[(int64_t)owner * a.W + r.tb / kPageTokens];
    if (page < 0 || page >= a.num_pages) {
      flag(a.status, MX4_STATUS_BAD_PAGE);
      return r;
    }
    r.page = page;
    const int64_t at = ((int64_t)page * a.Hkv + head) * kPageSubs + (r.tb % kPageTokens) / kSub;
    r.sc = a.ks[at] | (a.vs[at] << 8);
    return r;
  };

  const int n = (int)n64;
  Unit cur = resolve(lane), next = resolve(32 + lane);
  int issued = 0;
  bool dead = false;
  const uint32_t ring = smem_addr(sm) + group * S * kStepBytes;
  // unit k's rows into its stage (k < 32 ahead of the current chunk's first unit); one warp of the
  // group calls it
  auto issue = [&](int k, int chunk) {
    const bool in_next = k >= chunk + 32;
    const int page = __shfl_sync(0xFFFFFFFFu, in_next ? next.page : cur.page, k & 31);
    const int tb = __shfl_sync(0xFFFFFFFFu, in_next ? next.tb : cur.tb, k & 31);
    const int tile = __shfl_sync(0xFFFFFFFFu, in_next ? next.tile : cur.tile, k & 31);
    if (lane == 0) {
      const int st = k % S;
      const uint32_t bar = smem_addr(full + st), dst = ring + st * kStepBytes;
      if (page >= 0) {
        const int head = tile_of(a, tile).head;
        mbar_arrive_expect_tx(bar, kStepBytes);
        tensor_copy(dst, &a.kmap, tb % kPageTokens, head, page, bar);
        tensor_copy(dst + kSub * kFp8Row, &a.vmap, tb % kPageTokens, head, page, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    issued = k + 1;
  };
  if (wig == 0)
    for (int k = 0; k < min(S, n); ++k) issue(k, 0);

  Rows w;
  Tile tile{0, 0, 0};
  int tile_id = -1, head_id = -1, first = 0;
  bool active = false;  // this warp has rows of the tile
  // rows of scratch memory, of this warp and of the CTA's first
  const int64_t cta_row = (int64_t)blockIdx.x * kWarps * 16, my_row = cta_row + warp * 16 + (lane >> 2);
  float* const scratchmz = a.scratch + (int64_t)gridDim.x * kWarps * 16 * kHeadDim;
  float* const recmz = a.rec + 2 * (int64_t)gridDim.x * 16 * M * kHeadDim;

  auto out_row = [&](int h) {  // this lane's row g + 8 h: its number among the owner's rows
    return tile.rt * 16 * M + wig * 16 + (lane >> 2) + 8 * h;
  };
  auto write_out = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = out_row(h);
      if (r >= a.R) continue;
      const int64_t at = row_of<Lists>(a, tile, r);
      const float inv = w.z[h] == 0.f ? 0.f : 1.f / w.z[h];
      uint4* const p = reinterpret_cast<uint4*>(a.out + at * kHeadDim + 32 * (lane & 3));
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = 8 * i, x = 2 * h + e;
          p[2 * e + i] = make_uint4(bf16x2_bits(w.o[j][x] * inv, w.o[j + 1][x] * inv),
                                    bf16x2_bits(w.o[j + 2][x] * inv, w.o[j + 3][x] * inv),
                                    bf16x2_bits(w.o[j + 4][x] * inv, w.o[j + 5][x] * inv),
                                    bf16x2_bits(w.o[j + 6][x] * inv, w.o[j + 7][x] * inv));
        }
      if (a.lse && (lane & 3) == 0) a.lse[at] = row_lse(w.m[h], w.z[h]);
    }
  };

  // The pieces of tile id in this CTA: the last tiles of `cnt` groups from gi on, then the first tile
  // of group `tail` (-1: none).  to: 2 the result, else the piece of the CTA in rec.
  auto join = [&](int64_t id, int gi, int cnt, int tail, int to) {
    const Tile t = tile_of(a, id);
    for (int r = warp; r < 16 * M; r += kWarps) {
      const int row = t.rt * 16 * M + r;
      if (row >= a.R) continue;
      const float* const p = reinterpret_cast<const float*>(sm) + r * kRecRow;
      const int64_t tr = cta_row + tail * M * 16 + r;
      float m = tail >= 0 ? __ldcg(scratchmz + 2 * tr) : -INFINITY;
      for (int x = gi; x < gi + cnt; ++x)
        if (seg[3 * x] == id) m = fmaxf(m, p[x * 16 * M * kRecRow + kHeadDim]);
      const float ref = m == -INFINITY ? 0.f : m;
      float z = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = gi; x < gi + cnt; ++x) {
        const float* const y = p + x * 16 * M * kRecRow;
        if (seg[3 * x] == id)
          add_piece(acc, z, *reinterpret_cast<const float4*>(y + 4 * lane), y[kHeadDim], y[kHeadDim + 1], ref);
      }
      if (tail >= 0)
        add_piece(acc, z, __ldcg(reinterpret_cast<const float4*>(a.scratch + tr * kHeadDim) + lane),
                  __ldcg(scratchmz + 2 * tr), __ldcg(scratchmz + 2 * tr + 1), ref);
      if (to == 2) {
        put_row<Lists>(a, t, row, acc, m, z, lane);
      } else {
        const int64_t at = (2 * (int64_t)blockIdx.x + to) * 16 * M + r;
        *reinterpret_cast<float4*>(a.rec + at * kHeadDim + 4 * lane) = acc;
        if (lane == 0) *reinterpret_cast<float2*>(recmz + 2 * at) = make_float2(m, z);
      }
    }
  };

  int chunk = 0;
  for (int k = 0; k < n && !dead; ++k) {
    if (k - chunk == 32) {
      chunk = k;
      cur = next;
      next = resolve(k + 32 + lane);
    }
    const int id = __shfl_sync(0xFFFFFFFFu, cur.tile, k & 31);
    if (id != tile_id) {
      if (tile_id >= 0) {  // the tile in front ends inside this range: it is whole, or its last piece
        w.sum_z();
        if (first == 0) {
          if (active) write_out();
        } else {
          head_id = tile_id;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            w.put(h, a.scratch + (my_row + 8 * h) * kHeadDim, scratchmz + (my_row + 8 * h) * 2, lane);
        }
      }
      tile_id = id;
      tile = tile_of(a, id);
      first = __shfl_sync(0xFFFFFFFFu, cur.i, k & 31);
      const int s = Lists ? tile.owner / a.Q : tile.owner;
      const int base = a.seq_lens[s] - a.Q + (Lists ? tile.owner % a.Q : 0);
      const int r0 = tile.rt * 16 * M + wig * 16, r1 = min(r0 + 15, a.R - 1);
      active = r0 < a.R;
      w.clear();
      w.min_lim = Lists ? base : base + r0 / a.G;
      w.max_lim = Lists ? base : base + max(r1, 0) / a.G;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = out_row(h);
        const bool real = r < a.R;
        w.lim[h] = !real ? -1 : Lists ? base : base + r / a.G;
        w.load_q(a.q + (real ? row_of<Lists>(a, tile, r) : 0) * kHeadDim, real, h, a.scale, lane);
      }
    }
    const int tb = __shfl_sync(0xFFFFFFFFu, cur.tb, k & 31);
    const int page = __shfl_sync(0xFFFFFFFFu, cur.page, k & 31);
    const int sc = __shfl_sync(0xFFFFFFFFu, cur.sc, k & 31);
    const int st = k % S;
    if (!mbar_wait(smem_addr(full + st), (k / S) & 1)) dead = true;
    dead = __any_sync(0xFFFFFFFFu, dead);
    if (dead) {
      if (lane == 0) flag(a.status, MX4_STATUS_TIMEOUT);
      break;
    }
    if (page >= 0 && active) {
      const uint32_t ka = ring + st * kStepBytes, va = ka + kSub * kFp8Row;
      const float ek = e8m0_to_float(sc & 0xFF), ev = e8m0_to_float(sc >> 8);
      if (tb + kSub - 1 <= w.min_lim)
        w.template step<false>(ka, va, ek, ev, tb, lane);
      else
        w.template step<true>(ka, va, ek, ev, tb, lane);
    }
    __syncwarp();
    if (M == 1) {
      if (k + S < n) issue(k + S, chunk);
    } else {
      if (lane == 0) mbar_arrive(smem_addr(empty + st));
      if (wig == 0 && k >= 1 && k - 1 + S < n) {  // the stage before: the others are done by now
        const int e = k - 1;
        if (!mbar_wait(smem_addr(empty + e % S), (e / S) & 1)) dead = true;
        dead = __any_sync(0xFFFFFFFFu, dead);
        if (!dead)
          issue(e + S, chunk);
        else if (lane == 0)
          flag(a.status, MX4_STATUS_TIMEOUT);
      }
    }
  }
  // copies in flight land before their memory is used again (all have, but after a time-out)
  if (wig == 0 && lane == 0)
    for (int k = max(0, issued - S); k < issued; ++k)
      mbar_wait(smem_addr(full + k % S), (k / S) & 1);

  // ---- pieces: each group's last tile is in registers, a tile that it ended inside its range but
  // did not begin in the scratch memory.  Pieces of one tile are joined, in the order of the units.
  if (wig == 0 && lane == 0) {
    seg[3 * group] = n > 0 ? tile_id : -1;
    seg[3 * group + 1] = u0 + n;
    seg[3 * group + 2] = head_id;
  }
  if (n > 0) w.sum_z();
  __syncthreads();  // all stages are read
  float* const mine = reinterpret_cast<float*>(sm) + (warp * 16 + (lane >> 2)) * kRecRow;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w.put(h, mine + h * 8 * kRecRow, mine + h * 8 * kRecRow + kHeadDim, lane);
  if (tid == 0) a.meta[3 * blockIdx.x] = -1;
  __syncthreads();
  bool front = true;  // no group with units so far
  for (int gi = 0; gi < NG; ++gi) {
    if (seg[3 * gi] < 0) continue;
    if (front && seg[3 * gi + 2] >= 0)  // the end of a tile that began in a CTA before
      join(seg[3 * gi + 2], gi, 0, gi, 0);
    front = false;
    const int64_t id = seg[3 * gi];
    int prev = gi - 1, last = gi, behind;
    while (prev >= 0 && seg[3 * prev] < 0) --prev;
    if (prev >= 0 && seg[3 * prev] == id) continue;  // joined by the first group of the tile
    for (int x = gi + 1; x < NG; ++x)
      if (seg[3 * x] == id) last = x;
    for (behind = last + 1; behind < NG && seg[3 * behind] < 0;) ++behind;
    const bool ends = behind < NG && seg[3 * behind + 2] == id;
    const Tile t = tile_of(a, id);
    int64_t x0, x1;  // the tile's units
    if (Lists) {
      x0 = id * a.kb * kPageSubs;
      x1 = x0 + a.kb * kPageSubs;
    } else {
      const int64_t before = t.owner ? pref[t.owner - 1] : 0, units = pref[t.owner] - before;
      x0 = before * HR + (id - (int64_t)t.owner * HR) * units;
      x1 = x0 + units;
    }
    const bool begins = x0 >= cut.group_lo(blockIdx.x, gi, NG);
    const bool whole = begins && (ends || seg[3 * last + 1] == x1);
    join(id, gi, last - gi + 1, ends ? behind : -1, whole ? 2 : begins ? 1 : 0);
    if (begins && !whole && tid == 0) {  // the second kernel joins it with those of the next CTAs
      a.meta[3 * blockIdx.x] = id;
      a.meta[3 * blockIdx.x + 1] = (x1 - 1) / cut.per;
    }
  }
}

// Joins the pieces of the tiles that begin in CTA blockIdx.x of the first kernel and end in another:
// two rows a CTA, four warps each.
template <int M, bool Lists>
__global__ void __launch_bounds__(256) fp8_join_kernel(const __grid_constant__ DecodeArgs a, int ctas) {
  __shared__ float4 acc_s[8][32];
  __shared__ float2 mz_s[8];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t id = a.meta[3 * blockIdx.x];
  if (id < 0) return;
  const int last = (int)a.meta[3 * blockIdx.x + 1];
  const Tile t = tile_of(a, id);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & 3;
  const int r = 2 * blockIdx.y + (warp >> 2), row = t.rt * 16 * M + r;
  const float* const recmz = a.rec + 2 * (int64_t)ctas * 16 * M * kHeadDim;
  auto slot = [&](int x) {  // CTA x's piece: its last tile's, or the one that it began in
    return ((2 * (int64_t)x + (x == (int)blockIdx.x ? 1 : 0)) * 16 * M + r);
  };
  float m = -INFINITY, z = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < a.R) {
    for (int x = blockIdx.x + lane; x <= last; x += 32) m = fmaxf(m, recmz[2 * slot(x)]);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 8
    for (int x = blockIdx.x + part; x <= last; x += 4) {
      const float2 mz = *reinterpret_cast<const float2*>(recmz + 2 * slot(x));
      const float4 v = *reinterpret_cast<const float4*>(a.rec + slot(x) * kHeadDim + 4 * lane);
      add_piece(acc, z, v, mz.x, mz.y, ref);
    }
  }
  acc_s[warp][lane] = acc;
  if (lane == 0) mz_s[warp] = make_float2(m, z);
  __syncthreads();
  if (part != 0 || row >= a.R) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const float4 v = acc_s[warp + i][lane];
    z += mz_s[warp + i].y;
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  put_row<Lists>(a, t, row, acc, m, z, lane);
}

cudaError_t kv_map(const uint8_t* pages, int64_t page_stride, int64_t head_stride, int64_t num_pages,
                   int Hkv, CUtensorMap* tm) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {kFp8Row, kPageTokens, (cuuint64_t)Hkv, (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {kFp8Row, (cuuint64_t)(Hkv > 1 ? head_stride : kFp8Page),
                                 (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {kFp8Row, kSub, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(pages), dims,
                         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Workspace: pieces for the second kernel [2 CTAs][16 M][128], their m and z [2 CTAs][16 M][2],
// scratch of the groups [8 CTAs][16][128] and [8 CTAs][16][2], meta [CTAs][3].
size_t piece_floats(int rows_a_cta, int ctas) {
  return (size_t)ctas * (2 * rows_a_cta + kWarps * 16) * (kHeadDim + 2);
}
size_t ws_bytes(int M, int ctas) {
  return piece_floats(16 * M, ctas) * 4 + (size_t)ctas * 3 * sizeof(int64_t);
}

// Rows a tile: the fewest warps whose 16 rows each hold all rows of an owner, at most eight.
int warps_of(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 8; }

template <int M, bool Lists>
cudaError_t launch(DecodeArgs a, int64_t B, int num_sms, cudaStream_t stream) {
  auto kern = fp8_decode_kernel<M, Lists>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  a.RT = (a.R + 16 * M - 1) / (16 * M);
  a.scratch = a.rec + (size_t)num_sms * 2 * 16 * M * (kHeadDim + 2);
  a.meta = reinterpret_cast<int64_t*>(a.rec + piece_floats(16 * M, num_sms));
  const DecodeArgs all = a;
  const int64_t step = Lists ? B : kMaxOwners;  // lists take no prefix sums
  for (int64_t b0 = 0; b0 < B; b0 += step) {
    a = all;
    a.B = (int)std::min<int64_t>(step, B - b0);
    a.q += b0 * a.Q * a.H * kHeadDim;
    a.out += b0 * a.Q * a.H * kHeadDim;
    if (a.lse) a.lse += b0 * a.Q * a.H;
    a.table += b0 * a.W;
    a.seq_lens += b0;
    e = launch_pdl(kern, dim3(num_sms), dim3(kThreads), kSmemBytes, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(fp8_join_kernel<M, Lists>, dim3(num_sms, 8 * M), dim3(256), 0, stream, a, num_sms);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t fp8_decode_workspace_bytes(int rows, int num_sms) { return ws_bytes(warps_of(rows), num_sms); }

cudaError_t launch_fp8_decode(const uint16_t* q, int64_t B, int Q, int H, int Hkv,
                              const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
                              const uint8_t* v_scales, int64_t page_stride, int64_t head_stride,
                              int64_t num_pages, const int32_t* block_table, int64_t bt_width,
                              const int32_t* seq_lens, const int32_t* block_idx, int kb, float scale,
                              uint16_t* out, float* lse, void* ws, uint32_t* status, int num_sms,
                              cudaStream_t stream) {
  DecodeArgs a{};
  cudaError_t e = kv_map(k_pages, page_stride, head_stride, num_pages, Hkv, &a.kmap);
  if (e == cudaSuccess) e = kv_map(v_pages, page_stride, head_stride, num_pages, Hkv, &a.vmap);
  if (e != cudaSuccess) return e;
  a.q = q;
  a.ks = k_scales;
  a.vs = v_scales;
  a.table = block_table;
  a.W = bt_width;
  a.seq_lens = seq_lens;
  a.idx = block_idx;
  a.kb = kb;
  a.num_pages = num_pages;
  a.Q = Q;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.R = block_idx ? a.G : Q * a.G;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.rec = static_cast<float*>(ws);
  a.status = status;
  switch (warps_of(a.R)) {
    case 1: return block_idx ? launch<1, true>(a, B, num_sms, stream) : launch<1, false>(a, B, num_sms, stream);
    case 2: return block_idx ? launch<2, true>(a, B, num_sms, stream) : launch<2, false>(a, B, num_sms, stream);
    case 4: return block_idx ? launch<4, true>(a, B, num_sms, stream) : launch<4, false>(a, B, num_sms, stream);
    default: return block_idx ? launch<8, true>(a, B, num_sms, stream) : launch<8, false>(a, B, num_sms, stream);
  }
}

}  // namespace mx4
