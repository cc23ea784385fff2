// fp8_rope_append: new tokens' q and K heads turned by their positions, q out as bf16, K and V into
// the 8-bit cache.
//
// Turn.  Dims below R of a head form pairs (i, i + R/2), or (2 i, 2 i + 1); pair i turns by the
// angle position * w_i.  w_i comes in turns a position, as a 64-bit binary fraction: the product
// with the position wraps modulo one turn and is exact to 2^-64 * position turns, and goes to the sine
// as an fp32 number: positions of any size keep its 24 bits, small angles too.
//
// Store.  A block of 32 cached tokens of a head shares the scale 2^E, the smallest with
// amax <= 448 2^E (no value saturates), E >= -127.  Where E grows the block's stored codes are rounded
// to the new scale (a power of two moves E4M3's normal values without rounding).
//
// Work.  A decode step (fewer than eight new tokens a sequence on average): a warp a token and KV
// head, K and V, whose rows are on their way before the sequence is looked up.  Prompts: sixteen warps
// a block of 32 tokens, K or V, eight heads one after another, so that the sines of a token are
// computed once for eight heads.  q: a warp a token and 8 to 64 heads.  A lane computes the sines of two of its four dims; its partner in
// the pair has the others.
//
// Bound: latency for a decode batch, HBM for prompts.
#include <cuda_fp8.h>

#include "fp8_kv.cuh"

namespace mx4 {

namespace {

struct AppendArgs {
  const void* q;  // [T, H, 128] rows at q_stride elements a token (or null)
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  int64_t T;
  int H, Hkv;
  const int32_t* cu;         // [B + 1]: first new token of each sequence
  int B;
  const int64_t* positions;  // [T] or null: the position in the cache
  const uint64_t* phases;    // [R / 2] turns a position, in units of 2^-64
  int R;
  int interleaved;
  float factor;
  const int32_t* table;
  int64_t W;
  const int32_t* seq_lens;
  uint8_t* k_pages;
  uint8_t* v_pages;
  int64_t page_stride, head_stride, num_pages;
  uint8_t* ks;
  uint8_t* vs;
  uint16_t* q_out;
  int64_t kv_ctas;   // the q tasks (token, q_heads heads) follow them
  int q_heads;
  uint32_t* status;
};

constexpr int kQBatch = 8;   // q rows in flight
constexpr int kKvHeads = 8;  // heads of a prompt's block, one after another
constexpr int kPromptWarps = 16, kRows = kSub / kPromptWarps;  // and its rows

template <typename E>
__device__ __forceinline__ float4 load4(const E* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_bits_to_float(w.x & 0xFFFFu), bf16_bits_to_float(w.x >> 16),
                     bf16_bits_to_float(w.y & 0xFFFFu), bf16_bits_to_float(w.y >> 16));
}

// The sequence of new token t: cu[s] <= t < cu[s + 1]; -1 if none.  All lanes of a warp together:
// 32 probes a round.
__device__ __forceinline__ int sequence_of(const AppendArgs& a, int64_t t, int lane) {
  int lo = 0, n = a.B;  // the number of entries 1 .. B that are <= t is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int hits = __popc(__ballot_sync(0xFFFFFFFFu, a.cu[lo + min(n, (lane + 1) * step)] <= t));
    const int up = min(n, hits * step);
    n = hits == 32 ? 0 : min(n, up + step) - up - 1;
    lo += up;
  }
  return lo < a.B && a.cu[lo] <= t && t < a.cu[lo + 1] ? lo : -1;
}

// Cosines and sines of a token's position for the lane's dims 4 l .. 4 l + 3 (1 and 0 past R),
// the sine with the sign that it has in this dim.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn turn_of(const AppendArgs& a, int64_t pos, int lane) {
  Turn t;
  const int to = a.R / 8;  // neighbours: pairs 2 l, 2 l + 1.  halves: lanes l and l + R / 8, pairs 4 l .. 4 l + 3
  const bool in = 4 * lane < a.R, upper = lane >= to;
  const int i0 = a.interleaved ? 2 * lane : 4 * (upper ? lane - to : lane) + (upper ? 2 : 0);
  float c[2], s[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
    if (in) {
      const int64_t turns = (int64_t)((uint64_t)pos * a.phases[i0 + e]);  // of 2^-64
      sincospif((float)turns * 0x1p-63f, &s[e], &c[e]);
      c[e] *= a.factor;
      s[e] *= a.factor;
    }
  }
  if (a.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t.c[e] = c[e >> 1];
      t.s[e] = (e & 1) ? s[e >> 1] : -s[e >> 1];
    }
  } else {
    const int other = !in ? lane : upper ? lane - to : lane + to;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float oc = __shfl_sync(0xFFFFFFFFu, c[e], other), os = __shfl_sync(0xFFFFFFFFu, s[e], other);
      t.c[e] = upper ? oc : c[e];
      t.c[2 + e] = upper ? c[e] : oc;
      t.s[e] = upper ? os : -s[e];
      t.s[2 + e] = upper ? s[e] : -os;
    }
  }
  return t;
}

__device__ __forceinline__ float4 turned(const AppendArgs& a, float4 x, const Turn& t, int lane) {
  float4 y;  // the pair's other element
  if (a.interleaved) {
    y = make_float4(x.y, x.x, x.w, x.z);
  } else {
    const int to = a.R / 8, src = lane < to ? lane + to : lane < 2 * to ? lane - to : lane;
    y.x = __shfl_sync(0xFFFFFFFFu, x.x, src);
    y.y = __shfl_sync(0xFFFFFFFFu, x.y, src);
    y.z = __shfl_sync(0xFFFFFFFFu, x.z, src);
    y.w = __shfl_sync(0xFFFFFFFFu, x.w, src);
  }
  if (4 * lane >= a.R) return x;
  return make_float4(fmaf(x.x, t.c[0], y.x * t.s[0]), fmaf(x.y, t.c[1], y.y * t.s[1]),
                     fmaf(x.z, t.c[2], y.z * t.s[2]), fmaf(x.w, t.c[3], y.w * t.s[3]));
}

__device__ __forceinline__ uint32_t e4m3x4(float4 x) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four stored codes times 2^-d, d > 0, to the nearest code.  In f16, exact where the result is not
// below half of E4M3's smallest value (2^-9) by far; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4_down(uint32_t w, int d) {
  uint32_t h[2], r[2];
  e4m3x4_f16x2(w, h[0], h[1]);
  const uint32_t f = __half_as_ushort(__float2half_rn(ldexpf(1.f, -min(d, 24))));
  const uint32_t f2 = f | (f << 16);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), *reinterpret_cast<const __half2*>(&f2));
    r[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(y), __NV_SATFINITE, __NV_E4M3);
  }
  return r[0] | (r[1] << 16);
}

__device__ __forceinline__ uint32_t finite_bits(float x) {  // of |x|; 0 where not finite
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// The smallest E >= -127 with x <= 448 * 2^E, x the number of these bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, -127);
}

// Where a block's rows go: its first new row's place and scale in K's or V's pool.
struct Block {
  uint8_t* rows;   // the block's first row
  uint8_t* scale;
  int at;          // its first new row
};
__device__ __forceinline__ Block block_of(const AppendArgs& a, int64_t page, int64_t pos, int h, int which) {
  Block b;
  const int sub = (int)(pos % kPageTokens) / kSub;
  b.at = (int)(pos % kSub);
  b.rows = (which ? a.v_pages : a.k_pages) + page * a.page_stride + (int64_t)h * a.head_stride + sub * kSub * kFp8Row;
  b.scale = (which ? a.vs : a.ks) + (page * a.Hkv + h) * kPageSubs + sub;
  return b;
}

__device__ __forceinline__ uint32_t largest(float4 x) {
  return max(max(finite_bits(x.x), finite_bits(x.y)), max(finite_bits(x.z), finite_bits(x.w)));
}
__device__ __forceinline__ bool all_finite(float4 x) {
  return isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w);
}

// The block's exponent from the largest new value's bits and the stored scale byte (a scale of NaN,
// 255, counts as the smallest); rows stored before move to it, i0 of n threads.
__device__ __forceinline__ int grow(const Block& b, uint32_t top, int old, int i0, int n) {
  const int e_old = old == 255 ? -127 : old - 127;
  const int e = max(scale_exponent(top), b.at ? e_old : -127);
  if (b.at && e > e_old) {
    uint4* const p = reinterpret_cast<uint4*>(b.rows);
    for (int i = i0; i < b.at * (kFp8Row / 16); i += n) {
      uint4 w = p[i];
      w.x = e4m3x4_down(w.x, e - e_old);
      w.y = e4m3x4_down(w.y, e - e_old);
      w.z = e4m3x4_down(w.z, e - e_old);
      w.w = e4m3x4_down(w.w, e - e_old);
      p[i] = w;
    }
  }
  if (i0 == 0) *b.scale = (uint8_t)(e + 127);
  return e;
}

__device__ __forceinline__ void store_row(const Block& b, int row, float4 x, int e, int lane) {
  // 2^-e, e in [-127, 127] (above 120 where the stored scale is): 2^-127 is no normal number
  const float down = __uint_as_float(e < 127 ? (uint32_t)(127 - e) << 23 : 0x00400000u);
  uint32_t w = e4m3x4(make_float4(x.x * down, x.y * down, x.z * down, x.w * down));
  if (!isfinite(x.x)) w |= 0x7Fu;  // what is not finite is stored as NaN
  if (!isfinite(x.y)) w |= 0x7F00u;
  if (!isfinite(x.z)) w |= 0x7F0000u;
  if (!isfinite(x.w)) w |= 0x7F000000u;
  *reinterpret_cast<uint32_t*>(b.rows + (b.at + row) * kFp8Row + 4 * lane) = w;
}

// New tokens t .. of sequence s, from t on up to the end of their block: position, count, page (-1:
// none).  false: t belongs to no sequence, or to one that is skipped; `next` is then where to go on.
struct Span {
  int64_t pos, page, t0;
  int cnt;
};
__device__ __forceinline__ bool span_of(const AppendArgs& a, int64_t t, int lane, Span* sp, int64_t* next) {
  const int s = sequence_of(a, t, lane);
  if (s < 0) {  // before the first sequence, or behind the last
    const int64_t first = a.cu[0];
    *next = t < first ? first : a.T;
    return false;
  }
  const int64_t t0 = a.cu[s], t1 = a.cu[s + 1], L = a.seq_lens[s];
  if (t1 > a.T || L < t1 - t0 || L > a.W * kPageTokens) {
    if (lane == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    *next = t1;
    return false;
  }
  sp->t0 = t0;
  sp->pos = L - (t1 - t);
  sp->cnt = (int)min(t1 - t, (int64_t)kSub - sp->pos % kSub);
  const int32_t page = a.table[s * a.W + sp->pos / kPageTokens];
  sp->page = page >= 0 && page < a.num_pages ? page : -1;
  *next = t + sp->cnt;
  return true;
}

template <typename E>
__device__ __forceinline__ void turn_q(const AppendArgs& a, int64_t task, int lane) {
  const int per = (a.H + a.q_heads - 1) / a.q_heads;
  const int64_t t = task / per;
  if (t >= a.T) return;
  const int h0 = (int)(task - t * per) * a.q_heads, h1 = min(h0 + a.q_heads, a.H);
  const E* const src = static_cast<const E*>(a.q) + t * a.q_stride + 4 * lane;
  uint16_t* const dst = a.q_out + t * a.H * kHeadDim + 4 * lane;
  float4 x[kQBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kQBatch; ++i)
      x[i] = h + i < h1 ? load4<E>(src + (h + i) * kHeadDim) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(h0);  // (ahead of the look-up)
  const int s = sequence_of(a, t, lane);
  if (s < 0) return;
  const int64_t t1 = a.cu[s + 1], L = a.seq_lens[s];
  if (t1 > a.T || L < t1 - a.cu[s] || L > a.W * kPageTokens) return;  // (reported with its K)
  Turn turn;
  if (a.R > 0) turn = turn_of(a, a.positions ? a.positions[t] : L - (t1 - t), lane);
  for (int h = h0; h < h1; h += kQBatch) {
    if (h > h0) load(h);
#pragma unroll
    for (int i = 0; i < kQBatch; ++i) {
      if (h + i >= h1) break;
      const float4 y = a.R > 0 ? turned(a, x[i], turn, lane) : x[i];
      uint2 w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(y.y), "f"(y.x));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(y.w), "f"(y.z));
      *reinterpret_cast<uint2*>(dst + (h + i) * kHeadDim) = w;
    }
  }
}

// A decode step: a warp a new token and KV head.  The first new token of a block takes the others of
// its sequence in the block with it, two sweeps over them if there are any.
template <typename E>
__global__ void __launch_bounds__(128) fp8_append_step_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x >= a.kv_ctas) return turn_q<E>(a, (blockIdx.x - a.kv_ctas) * 4 + warp, lane);
  const int64_t task = (int64_t)blockIdx.x * 4 + warp, t = task / a.Hkv;
  if (t >= a.T) return;
  const int h = (int)(task - t * a.Hkv);
  const E* const src[2] = {static_cast<const E*>(a.k) + t * a.k_stride + h * kHeadDim + 4 * lane,
                           static_cast<const E*>(a.v) + t * a.v_stride + h * kHeadDim + 4 * lane};
  const int64_t stride[2] = {a.k_stride, a.v_stride};
  const float4 first[2] = {load4<E>(src[0]), load4<E>(src[1])};  // (ahead of the look-up)
  Span sp;
  int64_t next;
  if (!span_of(a, t, lane, &sp, &next)) return;
  if (t != sp.t0 && sp.pos % kSub != 0) return;  // its block's first new token has it
  if (sp.page < 0) {
    if (lane == 0) flag(a.status, MX4_STATUS_BAD_PAGE);
    return;
  }
  auto row = [&](int which, int r) {
    float4 x = r == 0 ? first[which] : load4<E>(src[which] + r * stride[which]);
    if (which == 0 && a.R > 0) x = turned(a, x, turn_of(a, a.positions ? a.positions[t + r] : sp.pos + r, lane), lane);
    return x;
  };
  bool ok = true;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const Block b = block_of(a, sp.page, sp.pos, h, which);
    const int old = b.at ? (int)*b.scale : 0;
    float4 x = row(which, 0);
    uint32_t top = largest(x);
    ok &= all_finite(x);
    for (int r = 1; r < sp.cnt; ++r) {
      const float4 y = row(which, r);
      top = max(top, largest(y));
      ok &= all_finite(y);
    }
    const int e = grow(b, __reduce_max_sync(0xFFFFFFFFu, top), old, lane, 32);
    store_row(b, 0, x, e, lane);
    for (int r = 1; r < sp.cnt; ++r) store_row(b, r, row(which, r), e, lane);
  }
  if (!__all_sync(0xFFFFFFFFu, ok) && lane == 0) flag(a.status, MX4_STATUS_BAD_VALUE);
}

// Prompts: a CTA 32 new tokens, K or V, kKvHeads heads; a warp two rows of a block (13600 tokens
// of 40 + 8 fp32 heads: 105 us; four rows, and so half the warps, 121; four heads 114, two 138).
template <typename E>
__global__ void __launch_bounds__(kPromptWarps * 32) fp8_append_kernel(const AppendArgs a) {
  __shared__ uint32_t top_s[2][kPromptWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x >= a.kv_ctas) return turn_q<E>(a, (blockIdx.x - a.kv_ctas) * kPromptWarps + warp, lane);
  const int groups = (a.Hkv + kKvHeads - 1) / kKvHeads;
  const int64_t chunk = blockIdx.x / (2 * groups);
  const int rest = (int)(blockIdx.x - chunk * 2 * groups), which = rest & 1;
  const int h0 = (rest >> 1) * kKvHeads, h1 = min(h0 + kKvHeads, a.Hkv);
  const int64_t stride = which ? a.v_stride : a.k_stride, end = min(a.T, (chunk + 1) * 32);
  bool ok = true;
  int turn_no = 0;
  for (int64_t t = chunk * 32, next; t < end; t = next) {
    Span sp;
    if (!span_of(a, t, lane, &sp, &next)) continue;
    if (t != sp.t0 && sp.pos % kSub != 0) continue;  // (the chunk before has this block)
    if (sp.page < 0) {
      if (threadIdx.x == 0) flag(a.status, MX4_STATUS_BAD_PAGE);
      continue;
    }
    const int r0 = warp * kRows, rows = min(kRows, sp.cnt - r0);  // of this warp
    Turn turn[kRows];
    const bool turns = which == 0 && a.R > 0;
    if (turns) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i < rows) turn[i] = turn_of(a, a.positions ? a.positions[t + r0 + i] : sp.pos + r0 + i, lane);
    }
    const E* const src =
        (which ? static_cast<const E*>(a.v) : static_cast<const E*>(a.k)) + (t + r0) * stride + 4 * lane;
    for (int h = h0; h < h1; ++h) {
      const Block b = block_of(a, sp.page, sp.pos, h, which);
      const int old = b.at ? (int)*b.scale : 0;
      float4 x[kRows];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) x[i] = i < rows ? load4<E>(src + i * stride + h * kHeadDim) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= rows) break;
        if (turns) x[i] = turned(a, x[i], turn[i], lane);
        top = max(top, largest(x[i]));
        ok &= all_finite(x[i]);
      }
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      uint32_t* const ts = top_s[turn_no++ & 1];
      if (lane == 0) ts[warp] = top;
      __syncthreads();  // (and all have read the stored scale; the next block's maxima go to the other row)
#pragma unroll
      for (int i = 0; i < kPromptWarps; ++i) top = max(top, ts[i]);
      const int e = grow(b, top, old, threadIdx.x, kPromptWarps * 32);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= rows) break;
        store_row(b, r0 + i, x[i], e, lane);
      }
    }
  }
  if (!__all_sync(0xFFFFFFFFu, ok) && lane == 0) flag(a.status, MX4_STATUS_BAD_VALUE);
}

template <typename E>
cudaError_t launch(AppendArgs a, int num_sms, cudaStream_t stream) {
  const bool prompts = a.T >= 8 * (int64_t)a.B;
  a.kv_ctas = prompts ? (a.T + 31) / 32 * 2 * ((a.Hkv + kKvHeads - 1) / kKvHeads) : (a.T * a.Hkv + 3) / 4;
  // more heads a q warp once there are warps enough: the sines are computed once for them
  a.q_heads = kQBatch;
  while (a.q_heads < 64 && a.q_heads < a.H && a.T * a.H / a.q_heads > 32 * (int64_t)num_sms) a.q_heads *= 2;
  const int warps = prompts ? kPromptWarps : 4;
  const int64_t q_ctas = a.q ? (a.T * ((a.H + a.q_heads - 1) / a.q_heads) + warps - 1) / warps : 0;
  return launch_pdl(prompts ? fp8_append_kernel<E> : fp8_append_step_kernel<E>,
                    dim3((unsigned)(a.kv_ctas + q_ctas)), dim3(warps * 32), 0, stream, a);
}

}  // namespace

cudaError_t launch_fp8_append(const void* q, const void* k, const void* v, int fp32, const int64_t* strides,
                              int64_t T, int H, int Hkv, const int32_t* cu, int64_t B,
                              const int64_t* positions, const int64_t* phases, int rot, int interleaved,
                              float factor, const int32_t* table, int64_t W, const int32_t* seq_lens,
                              uint8_t* k_pages, uint8_t* v_pages, int64_t page_stride, int64_t head_stride,
                              int64_t num_pages, uint8_t* k_scales, uint8_t* v_scales, uint16_t* q_out,
                              uint32_t* status, int num_sms, cudaStream_t stream) {
  AppendArgs a{q, k, v, strides[0], strides[1], strides[2], T, H, Hkv, cu, (int)B, positions,
               reinterpret_cast<const uint64_t*>(phases), rot, interleaved, factor, table, W, seq_lens,
               k_pages, v_pages, page_stride, head_stride, num_pages, k_scales, v_scales, q_out, 0, 0, status};
  return fp32 ? launch<float>(a, num_sms, stream) : launch<uint16_t>(a, num_sms, stream);
}

}  // namespace mx4
