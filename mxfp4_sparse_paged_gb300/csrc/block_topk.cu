// block_topk: for each decode token the k blocks with the largest scores among its n visible ones,
// the first and last few of them in any case; ties to the lower index, ascending, -1 padded.
//
// One CTA a token.  Scores become integers of the same order (score_key), those always taken the
// largest.  Rows of up to 4096 blocks live in registers, consecutive blocks in a thread: the k-th
// largest key is built from its top bit down, two bits a round, counting the keys that reach each of
// three candidates; the start is the keys' common prefix.  One scan over the threads then gives
// every taken block its place.  Longer rows are cut to the keys that matter first: a histogram over
// equal steps of the score between the row's smallest and largest finds the step that holds the
// k-th, and only that step's keys are searched, in shared memory.
// Bound: latency (a row of 1024 scores is 4 KB).
#include "score_pipeline.cuh"

namespace mx4 {

namespace {

struct TopArgs {
  const float* scores;
  int64_t ld;
  const int32_t* seq_lens;
  int Q, k, first, last;
  int32_t* idx;
  uint32_t* status;
};

constexpr uint32_t kAlways = 0xFFFFFFFFu;  // above every score's key

__device__ __forceinline__ uint32_t order_key(float x) { return x != x ? kNanKey : score_key(x); }

// Sum over the CTA of a value whose total stays below 2^32, in every thread.
template <int THREADS>
__device__ __forceinline__ uint32_t cta_sum(uint32_t v, uint32_t* buf, int& turn) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  uint32_t* const b = buf + (turn ^= 1) * (THREADS / 32);
  if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t s = 0;
  if (THREADS <= 256) {
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) s += b[i];
  } else {
    s = __reduce_add_sync(0xFFFFFFFFu, b[threadIdx.x & (THREADS / 32 - 1)]);
  }
  return s;
}

// Exclusive prefix of a packed pair over the CTA's threads.
template <int THREADS>
__device__ __forceinline__ uint64_t cta_prefix(uint64_t v, uint64_t* buf, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  uint64_t before = inc - v, all = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += buf[i];
    all += buf[i];
  }
  *total = all;
  return before;
}

// The largest key that at least `want` (>= 1) of the CTA's keys reach, and how many exceed it.
// get(i) for i < PER are the thread's keys; keys of 0 stand for none.
template <int THREADS, int PER, class Get>
__device__ __forceinline__ uint32_t kth_key(Get get, uint32_t want, uint32_t* buf, int& turn, uint32_t* above) {
  uint32_t key = 0, over = 0;  // over: keys above the candidates with this prefix
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = key | (1u << bit);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += get(i) >= cand;
    c = cta_sum<THREADS>(c, buf, turn);
    if (c >= want) key = cand; else over = c;
  }
  *above = over;
  return key;
}

template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) block_topk_kernel(const TopArgs a) {
  __shared__ uint32_t buf[2 * (THREADS / 32)];
  __shared__ uint64_t buf64[THREADS / 32];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  int turn = 0;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t L = a.seq_lens[t / a.Q], p = L - a.Q + t % a.Q;
  int32_t* const out = a.idx + t * a.k;
  int n = p >= 0 ? (int)(p / kPageTokens) + 1 : 0;
  if (L < 0 || n > a.ld) {
    if (tid == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    n = 0;
  }
  const int k = min(a.k, n);
  for (int i = k + tid; i < a.k; i += THREADS) out[i] = -1;
  if (k == n) {
    for (int i = tid; i < n; i += THREADS) out[i] = i;
    return;
  }
  const float* const x = a.scores + t * a.ld;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    key[i] = b >= n ? 0u : b < a.first || b >= n - a.last ? kAlways : order_key(x[b]);
  }
  uint32_t above;
  const uint32_t kth = kth_key<THREADS, PER>([&](int i) { return key[i]; }, k, buf, turn, &above);
  uint64_t mine = 0, total;  // keys above the k-th, and equal to it
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += (key[i] > kth ? 1ull << 32 : 0ull) + (key[i] == kth ? 1ull : 0ull);
  const uint64_t before = cta_prefix<THREADS>(mine, buf64, &total);
  const uint32_t ties = k - above;
  uint32_t gt = (uint32_t)(before >> 32), eq = (uint32_t)before;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t at = gt + min(eq, ties);
    if (key[i] > kth || (key[i] == kth && eq < ties)) out[at] = tid * PER + i;
    gt += key[i] > kth;
    eq += key[i] == kth;
  }
}

// Rows of more than 4096 blocks.
constexpr int kBins = 4096;
constexpr int kLongThreads = 1024;
constexpr int kCands = 8192;  // keys of the step that holds the k-th (more: all keys are searched)
struct LongSmem {
  uint32_t hist[kBins];
  uint32_t cand[kCands];
  uint32_t buf[2 * (kLongThreads / 32)];
  uint64_t buf64[kLongThreads / 32];
  float lo[kLongThreads / 32], hi[kLongThreads / 32];
  uint32_t n_cand, bin, above;
};

__global__ void __launch_bounds__(kLongThreads) block_topk_long_kernel(const TopArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  LongSmem& s = *reinterpret_cast<LongSmem*>(smem);
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int turn = 0;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t L = a.seq_lens[t / a.Q], p = L - a.Q + t % a.Q;
  int32_t* const out = a.idx + t * a.k;
  int n = p >= 0 ? (int)(p / kPageTokens) + 1 : 0;
  if (L < 0 || n > a.ld) {
    if (tid == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    n = 0;
  }
  const int k = min(a.k, n);
  for (int i = k + tid; i < a.k; i += kLongThreads) out[i] = -1;
  if (k == n) {
    for (int i = tid; i < n; i += kLongThreads) out[i] = i;
    return;
  }
  const float* const x = a.scores + t * a.ld;
  auto key_of = [&](int b) { return b < a.first || b >= n - a.last ? kAlways : order_key(x[b]); };

  // ---- the range of the finite scores
  float lo = INFINITY, hi = -INFINITY;
  for (int i = tid; i < kBins; i += kLongThreads) s.hist[i] = 0;
#pragma unroll 8
  for (int b = tid; b < n; b += kLongThreads) {
    const float v = x[b];
    if (isfinite(v)) {
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
  }
  if (lane == 0) {
    s.lo[warp] = lo;
    s.hi[warp] = hi;
  }
  if (tid == 0) s.n_cand = 0;
  __syncthreads();
  lo = s.lo[lane];
  hi = s.hi[lane];
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
  }
  // a step's number never falls as the key grows: both are monotone in the score
  const float w = hi > lo ? (float)(kBins - 3) / (hi - lo) : 0.f;
  auto bin_of = [&](float v) {
    if (v != v || v == INFINITY) return kBins - 1;
    if (v == -INFINITY) return 0;
    const float f = (v - lo) * w;  // (a range beyond fp32, or one too small to divide by, is one step)
    return 1 + (f < (float)(kBins - 3) ? (int)f : kBins - 3);
  };
  auto bin_at = [&](int b) { return b < a.first || b >= n - a.last ? kBins - 1 : bin_of(x[b]); };
#pragma unroll 4
  for (int b = tid; b < n; b += kLongThreads) atomicAdd(&s.hist[bin_at(b)], 1u);
  __syncthreads();

  // ---- the step that holds the k-th: thread i has steps 4 i .. 4 i + 3 counted from the top
  {
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += c[i] = s.hist[kBins - 1 - (4 * tid + i)];
    uint64_t total;
    uint32_t before = (uint32_t)cta_prefix<kLongThreads>(sum, s.buf64, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before < (uint32_t)k && before + c[i] >= (uint32_t)k) {
        s.bin = kBins - 1 - (4 * tid + i);
        s.above = before;
      }
      before += c[i];
    }
  }
  __syncthreads();
  const int bin = s.bin;
  const uint32_t over = s.above, held = s.hist[bin];

  // ---- the k-th key
  uint32_t kth, above;
  if (held <= kCands) {
#pragma unroll 4
    for (int b = tid; b < n; b += kLongThreads)
      if (bin_at(b) == bin) s.cand[atomicAdd(&s.n_cand, 1u)] = key_of(b);
    __syncthreads();
    uint32_t key[kCands / kLongThreads];
#pragma unroll
    for (int i = 0; i < kCands / kLongThreads; ++i)
      key[i] = i * kLongThreads + tid < (int)held ? s.cand[i * kLongThreads + tid] : 0u;
    kth = kth_key<kLongThreads, kCands / kLongThreads>([&](int i) { return key[i]; }, k - over, s.buf, turn, &above);
    above += over;
  } else {
    kth = 0, above = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = kth | (1u << bit);
      uint32_t c = 0;
#pragma unroll 4
      for (int b = tid; b < n; b += kLongThreads) c += key_of(b) >= cand;
      c = cta_sum<kLongThreads>(c, s.buf, turn);
      if (c >= (uint32_t)k) kth = cand; else above = c;
    }
  }

  // ---- taken blocks to their places, a tile of 4 a thread at a time
  const uint32_t ties = k - above;
  uint32_t gt0 = 0, eq0 = 0;
  for (int base = 0; base < n && gt0 + min(eq0, ties) < (uint32_t)k; base += 4 * kLongThreads) {
    uint32_t key[4];
    uint64_t mine = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = base + 4 * tid + i;
      key[i] = b < n ? key_of(b) : 0u;
      if (b < n) mine += (key[i] > kth ? 1ull << 32 : 0ull) + (key[i] == kth ? 1ull : 0ull);
    }
    const uint64_t before = cta_prefix<kLongThreads>(mine, s.buf64, &total);
    uint32_t gt = gt0 + (uint32_t)(before >> 32), eq = eq0 + (uint32_t)before;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = base + 4 * tid + i;
      if (b >= n) break;
      if (key[i] > kth || (key[i] == kth && eq < ties)) out[gt + min(eq, ties)] = b;
      gt += key[i] > kth;
      eq += key[i] == kth;
    }
    gt0 += (uint32_t)(total >> 32);
    eq0 += (uint32_t)total;
  }
}

}  // namespace

cudaError_t launch_block_topk(const float* scores, int64_t ld, const int32_t* seq_lens, int64_t T, int q,
                              int k, int first, int last, int32_t* idx, uint32_t* status,
                              cudaStream_t stream) {
  const TopArgs a{scores, ld, seq_lens, q, k, first, last, idx, status};
  const dim3 grid((unsigned)T);
  if (ld <= 1024) return launch_pdl(block_topk_kernel<256, 4>, grid, dim3(256), 0, stream, a);
  if (ld <= 4096) return launch_pdl(block_topk_kernel<256, 16>, grid, dim3(256), 0, stream, a);
  cudaError_t e = cudaFuncSetAttribute(block_topk_long_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(LongSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(block_topk_long_kernel, grid, dim3(kLongThreads), sizeof(LongSmem), stream, a);
}

}  // namespace mx4
