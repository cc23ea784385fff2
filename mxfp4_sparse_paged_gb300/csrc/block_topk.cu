// block_topk: for each decode token the k blocks with the largest scores among its n visible ones,
// the first and last few of them in any case; ties to the lower index, ascending, -1 padded.
//
// A CTA a token, or a cluster of eight where a row has more than 4096 blocks.  Scores become integers
// of the same order (score_key), those always taken the largest, and stay in registers, consecutive
// blocks in a thread.  The k-th largest key is found byte by byte from the top: a histogram of the
// keys that still match in shared memory (a cluster adds up its CTAs' histograms through distributed
// shared memory, every CTA for itself), and the byte at which the count from above reaches k.  One
// scan over the threads (and the CTAs' counts) then gives every taken block its place.
// Bound: latency.  A row of 1024 scores is 4 KB; one of 65536 took a single CTA that went through it
// five times 80 us.
#include <cooperative_groups.h>

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

template <int THREADS, int PER, int CL>
__global__ void __launch_bounds__(THREADS) block_topk_kernel(const TopArgs a) {
  namespace cg = cooperative_groups;
  __shared__ uint32_t hist[2][256];
  __shared__ uint64_t buf64[THREADS / 32];
  __shared__ uint32_t byte_s, above_s;
  __shared__ uint64_t count_s;  // of this CTA: keys above the k-th, and equal to it
  const int64_t t = blockIdx.x / CL;
  const int tid = threadIdx.x, rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t s = t / a.Q, L = a.seq_lens[s], p = L - a.Q + (t - s * a.Q);
  int32_t* const out = a.idx + t * a.k;
  int n = p >= 0 ? (int)(p / kPageTokens) + 1 : 0;
  if (L < 0 || n > a.ld) {
    if (tid == 0 && rank == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    n = 0;
  }
  const int k = min(a.k, n);
  const int me = rank * THREADS + tid;
  for (int i = k + me; i < a.k; i += CL * THREADS) out[i] = -1;
  if (k == n) {  // (all CTAs of the cluster alike)
    for (int i = me; i < n; i += CL * THREADS) out[i] = i;
    return;
  }
  const float* const x = a.scores + t * a.ld;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = me * PER + i;
    key[i] = b >= n ? 0u : b < a.first || b >= n - a.last ? kAlways : order_key(x[b]);
  }
  uint32_t kth = 0, above = 0;  // keys that match kth's known bytes come after `above` larger ones
#pragma unroll
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    uint32_t* const h = hist[round & 1];
    if (tid < 256) h[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)  // (a key of 0 is none)
      if (key[i] != 0u && (round == 0 || (key[i] >> (shift + 8)) == (kth >> (shift + 8))))
        atomicAdd(&h[(key[i] >> shift) & 255u], 1u);
    // the histogram before the last one is read by no CTA any more once all are here
    if (CL > 1) cg::this_cluster().sync(); else __syncthreads();
    uint32_t c = 0;  // thread i has byte 255 - i
    if (tid < 256) {
      if (CL > 1) {
#pragma unroll
        for (int r = 0; r < CL; ++r) c += *cg::this_cluster().map_shared_rank(&h[255 - tid], r);
      } else {
        c = h[255 - tid];
      }
    }
    uint64_t total;
    const uint32_t before = above + (uint32_t)cta_prefix<THREADS>(c, buf64, &total);
    if (before < (uint32_t)k && before + c >= (uint32_t)k) {  // one thread
      byte_s = 255 - tid;
      above_s = before;
    }
    __syncthreads();
    kth |= byte_s << shift;
    above = above_s;
  }
  uint64_t mine = 0, total;  // keys above the k-th, and equal to it
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += (key[i] > kth ? 1ull << 32 : 0ull) + (key[i] == kth ? 1ull : 0ull);
  uint64_t before = cta_prefix<THREADS>(mine, buf64, &total);
  if (CL > 1) {
    if (tid == 0) count_s = total;
    cg::this_cluster().sync();
    for (int r = 0; r < rank; ++r) before += *cg::this_cluster().map_shared_rank(&count_s, r);
  }
  const uint32_t ties = k - above;
  uint32_t gt = (uint32_t)(before >> 32), eq = (uint32_t)before;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (key[i] > kth || (key[i] == kth && eq < ties)) out[gt + min(eq, ties)] = me * PER + i;
    gt += key[i] > kth;
    eq += key[i] == kth;
  }
  if (CL > 1) cg::this_cluster().sync();  // no CTA ends while another reads its counts
}

constexpr int kCluster = 8;

}  // namespace

cudaError_t launch_block_topk(const float* scores, int64_t ld, const int32_t* seq_lens, int64_t T, int q,
                              int k, int first, int last, int32_t* idx, uint32_t* status,
                              cudaStream_t stream) {
  const TopArgs a{scores, ld, seq_lens, q, k, first, last, idx, status};
  const dim3 grid((unsigned)T);
  if (ld <= 1024) return launch_pdl(block_topk_kernel<256, 4, 1>, grid, dim3(256), 0, stream, a);
  if (ld <= 4096) return launch_pdl(block_topk_kernel<256, 16, 1>, grid, dim3(256), 0, stream, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(T * kCluster));
  cfg.blockDim = dim3(512);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {kCluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, block_topk_kernel<512, 16, kCluster>, a);
}

}  // namespace mx4
