// fp8_rope_append: new tokens' q and K heads turned by their positions, q out as bf16, K and V into
// the 8-bit cache.
//
// Turn.  Dims below R of a head form pairs (i, i + R/2), or (2 i, 2 i + 1); pair i turns by the
// angle position * w_i.  w_i comes in turns a position, as a 64-bit binary fraction: the product
// with the position wraps modulo one turn and is exact to 2^-64 * position turns, so positions of
// any size keep all bits that an fp32 angle in [-pi, pi) holds.
//
// Store.  A block of 32 cached tokens of a head shares the scale 2^E, the smallest with
// amax <= 448 2^E (no value saturates), E >= -127.  One warp, or four where a sequence brings eight
// new tokens or more on average (one warp goes through 32 rows twice: once for the largest, once to
// store), takes the new rows of one block of K or V.  Where E grows the block's stored codes are
// rounded to the new scale.  A power of two moves E4M3's normal values without rounding.
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
  int64_t kv_tasks;  // (tokens, head, K or V); the q tasks (token, 8 heads) follow
  uint32_t* status;
};

constexpr int kQHeads = 8;  // heads that share a token's sines

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
  const int half = a.R / 2;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = 4 * lane + e;
    t.c[e] = 1.f;
    t.s[e] = 0.f;
    if (d < a.R) {
      const int i = a.interleaved ? d >> 1 : d < half ? d : d - half;
      const bool upper = a.interleaved ? d & 1 : d >= half;
      const int32_t turns = (int32_t)(((uint64_t)pos * a.phases[i]) >> 32);  // of 2^-32
      float s, c;
      sincospif((float)turns * 0x1p-31f, &s, &c);
      t.c[e] = c * a.factor;
      t.s[e] = upper ? s * a.factor : -s * a.factor;
    }
  }
  return t;
}

__device__ __forceinline__ float4 turned(const AppendArgs& a, float4 x, const Turn& t, int lane) {
  if (a.R == 0) return x;
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

// The rows of one block: cnt new rows from token t on, at row `at` of the block, of K (which = 0)
// or V of head h; NW warps together, this one the wig-th.
template <typename E, int NW>
__device__ __forceinline__ void store_block(const AppendArgs& a, int64_t t, int cnt, int64_t pos0, int64_t page,
                                            int h, int which, int wig, int lane, uint32_t* top_s) {
  constexpr int kBatch = 8;
  const E* const src = which ? static_cast<const E*>(a.v) + t * a.v_stride : static_cast<const E*>(a.k) + t * a.k_stride;
  const int64_t stride = which ? a.v_stride : a.k_stride;
  uint8_t* const pages = (which ? a.v_pages : a.k_pages) + page * a.page_stride + (int64_t)h * a.head_stride;
  const int at = (int)(pos0 % kSub), first = (int)(pos0 % kPageTokens);  // row of the block, of the page
  uint8_t* const scale = (which ? a.vs : a.ks) + (page * a.Hkv + h) * kPageSubs + first / kSub;
  float4 x[kBatch];
  auto rows = [&](int b) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      x[i] = b + i < cnt ? load4<E>(src + (b + i) * stride + h * kHeadDim + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (which == 0 && a.R > 0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (b + i >= cnt) break;
        x[i] = turned(a, x[i], turn_of(a, a.positions ? a.positions[t + b + i] : pos0 + b + i, lane), lane);
      }
    }
  };
  const int old = at ? (int)*scale : 0;
  uint32_t top = 0;
  bool bad = false;
  for (int b = wig * kBatch; b < cnt; b += NW * kBatch) {
    rows(b);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      top = max(top, max(max(finite_bits(x[i].x), finite_bits(x[i].y)), max(finite_bits(x[i].z), finite_bits(x[i].w))));
      bad |= !(isfinite(x[i].x) && isfinite(x[i].y) && isfinite(x[i].z) && isfinite(x[i].w));
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) flag(a.status, MX4_STATUS_BAD_VALUE);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (NW > 1) {
    __syncthreads();  // the block before has read its maxima
    if (lane == 0) top_s[wig] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) top = max(top, top_s[i]);
  }
  // stored rows keep their scale or get a larger one; a scale of NaN (255) counts as the smallest
  const int e_old = old == 255 ? -127 : old - 127;
  const int e = max(scale_exponent(top), at ? e_old : -127);
  if (at && e > e_old) {
    uint4* const p = reinterpret_cast<uint4*>(pages + (first - at) * kFp8Row);
    for (int i = wig * 32 + lane; i < at * (kFp8Row / 16); i += NW * 32) {
      uint4 w = p[i];
      w.x = e4m3x4_down(w.x, e - e_old);
      w.y = e4m3x4_down(w.y, e - e_old);
      w.z = e4m3x4_down(w.z, e - e_old);
      w.w = e4m3x4_down(w.w, e - e_old);
      p[i] = w;
    }
  }
  if (wig == 0 && lane == 0) *scale = (uint8_t)(e + 127);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, e in [-127, 120]
  for (int b = wig * kBatch; b < cnt; b += NW * kBatch) {
    if (cnt > NW * kBatch) rows(b);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (b + i >= cnt) break;
      float4 y = x[i];
      y = make_float4(y.x * down, y.y * down, y.z * down, y.w * down);
      uint32_t w = e4m3x4(y);
      if (bad) {  // what is not finite is stored as NaN
        if (!isfinite(x[i].x)) w |= 0x7Fu;
        if (!isfinite(x[i].y)) w |= 0x7F00u;
        if (!isfinite(x[i].z)) w |= 0x7F0000u;
        if (!isfinite(x[i].w)) w |= 0x7F000000u;
      }
      *reinterpret_cast<uint32_t*>(pages + (first + b + i) * kFp8Row + 4 * lane) = w;
    }
  }
}

// NW = 1: a warp a task, one token's chance to be its block's first new one.  NW = 4: a CTA a task,
// 32 tokens.
template <typename E, int NW>
__global__ void __launch_bounds__(128) fp8_append_kernel(const AppendArgs a) {
  constexpr int kTokens = NW == 1 ? 1 : 32;
  __shared__ uint32_t top_s[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t kv_ctas = NW == 1 ? (a.kv_tasks + 3) / 4 : a.kv_tasks;
  if (blockIdx.x < kv_ctas) {
    const int64_t task = NW == 1 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
    if (task >= a.kv_tasks) return;
    const int per = 2 * a.Hkv;
    const int64_t chunk = task / per;
    const int hw = (int)(task - chunk * per), h = hw >> 1, which = hw & 1;
    const int64_t end = min(a.T, (chunk + 1) * kTokens);
    for (int64_t t = chunk * kTokens; t < end;) {
      const int s = sequence_of(a, t, lane);
      if (s < 0) {  // before the first sequence, or behind the last
        if (t >= a.cu[0]) return;
        t = a.cu[0];
        continue;
      }
      const int64_t t0 = a.cu[s], t1 = a.cu[s + 1], L = a.seq_lens[s];
      if (t1 > a.T || L < t1 - t0 || L > a.W * kPageTokens) {
        if (lane == 0) flag(a.status, MX4_STATUS_BAD_LEN);
        t = t1;
        continue;
      }
      const int64_t pos = L - (t1 - t);
      const int cnt = (int)min(t1 - t, (int64_t)kSub - pos % kSub);
      if (t == t0 || pos % kSub == 0) {
        const int32_t page = a.table[s * a.W + pos / kPageTokens];
        if (page >= 0 && page < a.num_pages)
          store_block<E, NW>(a, t, cnt, pos, page, h, which, NW == 1 ? 0 : warp, lane, top_s);
        else if (lane == 0)
          flag(a.status, MX4_STATUS_BAD_PAGE);
      }
      t += cnt;
    }
    return;
  }
  const int per = (a.H + kQHeads - 1) / kQHeads;
  const int64_t task = (blockIdx.x - kv_ctas) * 4 + warp, t = task / per;
  if (t >= a.T) return;
  const int s = sequence_of(a, t, lane);
  if (s < 0) return;
  const int64_t t1 = a.cu[s + 1], L = a.seq_lens[s];
  if (t1 > a.T || L < t1 - a.cu[s] || L > a.W * kPageTokens) return;  // (reported with its K)
  Turn turn;
  if (a.R > 0) turn = turn_of(a, a.positions ? a.positions[t] : L - (t1 - t), lane);
  const int h0 = (int)(task - t * per) * kQHeads;
  const E* const src = static_cast<const E*>(a.q) + t * a.q_stride + 4 * lane;
  uint16_t* const dst = a.q_out + t * a.H * kHeadDim + 4 * lane;
  float4 x[kQHeads];
#pragma unroll
  for (int i = 0; i < kQHeads; ++i)
    x[i] = h0 + i < a.H ? load4<E>(src + (h0 + i) * kHeadDim) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kQHeads; ++i) {
    if (h0 + i >= a.H) break;
    const float4 y = turned(a, x[i], turn, lane);
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(y.y), "f"(y.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(y.w), "f"(y.z));
    *reinterpret_cast<uint2*>(dst + (h0 + i) * kHeadDim) = w;
  }
}

template <typename E>
cudaError_t launch(AppendArgs a, cudaStream_t stream) {
  const bool wide = a.T >= 8 * (int64_t)a.B;
  const int64_t q_ctas = a.q ? (a.T * ((a.H + kQHeads - 1) / kQHeads) + 3) / 4 : 0;
  a.kv_tasks = (wide ? (a.T + 31) / 32 : a.T) * 2 * a.Hkv;
  const int64_t grid = (wide ? a.kv_tasks : (a.kv_tasks + 3) / 4) + q_ctas;
  return launch_pdl(wide ? fp8_append_kernel<E, 4> : fp8_append_kernel<E, 1>, dim3((unsigned)grid), dim3(128), 0,
                    stream, a);
}

}  // namespace

cudaError_t launch_fp8_append(const void* q, const void* k, const void* v, int fp32, const int64_t* strides,
                              int64_t T, int H, int Hkv, const int32_t* cu, int64_t B,
                              const int64_t* positions, const int64_t* phases, int rot, int interleaved,
                              float factor, const int32_t* table, int64_t W, const int32_t* seq_lens,
                              uint8_t* k_pages, uint8_t* v_pages, int64_t page_stride, int64_t head_stride,
                              int64_t num_pages, uint8_t* k_scales, uint8_t* v_scales, uint16_t* q_out,
                              uint32_t* status, cudaStream_t stream) {
  AppendArgs a{q, k, v, strides[0], strides[1], strides[2], T, H, Hkv, cu, (int)B, positions,
               reinterpret_cast<const uint64_t*>(phases), rot, interleaved, factor, table, W, seq_lens,
               k_pages, v_pages, page_stride, head_stride, num_pages, k_scales, v_scales, q_out, 0, status};
  return fp32 ? launch<float>(a, stream) : launch<uint16_t>(a, stream);
}

}  // namespace mx4
