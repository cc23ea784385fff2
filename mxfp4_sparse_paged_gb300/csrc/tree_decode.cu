// tree_paged_decode: attention of a speculative step's nodes over the MXFP4 pages.
//
// One CTA per (sequence, KV head, 16 rows): a row is one (node, query head of the group)
// pair.  Pages are dequantised to fp32 in shared memory one at a time; a warp takes
// four rows, each lane four tokens of the page for the logits and four dims for the
// output, with one online softmax per row.
#include <cuda_bf16.h>

#include "common.cuh"

namespace mx4 {

constexpr int kRows = 16, kTreeWarps = 4;
constexpr int kPitch = kHeadDim + 1;

struct TreeArgs {
  const uint16_t* q;
  int N, H, Hkv;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  int64_t page_stride, head_stride, num_pages;
  const int32_t* table;
  int64_t bt_width;
  const int32_t* seq_lens;
  const int32_t* n_nodes;
  const uint64_t* mask;
  int64_t window, sinks;
  float scale;
  uint16_t* out;
  float* lse;
  uint32_t* status;
};

__global__ void __launch_bounds__(kTreeWarps * 32) tree_simple_kernel(const TreeArgs a) {
  extern __shared__ float sm[];
  float* sk = sm;                       // [128][129]
  float* sv = sk + kPageTokens * kPitch;
  float* sq = sv + kPageTokens * kPitch;  // [16][128]
  float* sp = sq + kRows * kHeadDim;      // [4 warps][128]
  __shared__ uint64_t s_mask[64];
  __shared__ int s_depth[64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t s = blockIdx.z;
  const int h = blockIdx.y, G = a.H / a.Hkv;
  const int r0 = blockIdx.x * kRows;
  pdl_launch_dependents();
  pdl_wait();
  int n = a.n_nodes ? a.n_nodes[s] : a.N;
  const int64_t L = a.seq_lens[s];
  if (n < 0 || n > a.N || L < n || L > a.bt_width * kPageTokens) {
    if (tid == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    n = 0;
  }
  const int64_t base = L - n;
  if (tid < n) {
    uint64_t m = a.mask ? a.mask[s * a.N + tid] : (2ull << tid) - 1;
    if (n < 64) m &= (1ull << n) - 1;
    s_mask[tid] = m;
    s_depth[tid] = max(1, __popcll(m)) - 1;
  }
  for (int e = tid; e < kRows * kHeadDim; e += blockDim.x) {
    const int r = r0 + e / kHeadDim, j = r / G, g = r % G;
    sq[e] = j < n ? bf16_bits_to_float(a.q[((s * a.N + j) * a.H + h * G + g) * kHeadDim +
                                           e % kHeadDim]) * a.scale
                  : 0.f;
  }
  __syncthreads();
  float m[4], l[4], o[4][4];
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    for (int d = 0; d < 4; ++d) o[i][d] = 0.f;
  }
  const bool any = r0 / G < n;
  const int64_t lo = a.window > 0 ? max((int64_t)0, base + 1 - a.window) : 0;
  for (int64_t pg = 0; any && pg * kPageTokens < L; ++pg) {
    if (a.window > 0 && (pg + 1) * kPageTokens <= lo && pg * kPageTokens >= a.sinks) continue;
    const int32_t pid = a.table[s * a.bt_width + pg];
    if (pid < 0 || pid >= a.num_pages) {
      if (tid == 0) flag(a.status, MX4_STATUS_BAD_PAGE);
      continue;
    }
    __syncthreads();
    for (int e = tid; e < 2 * kPageTokens * 16; e += blockDim.x) {
      const int which = e / (kPageTokens * 16), x = e % (kPageTokens * 16), row = x / 16, w = x % 16;
      const uint8_t* p = (which ? a.v_pages : a.k_pages) + pid * a.page_stride + h * a.head_stride;
      const uint32_t c = reinterpret_cast<const uint32_t*>(p + row * kRowDataBytes)[w];
      const float f = e8m0_to_float(p[kScaleOffset + row * kRowScaleBytes + w / 4]);
      float* dst = (which ? sv : sk) + row * kPitch + w * 8;
      for (int i = 0; i < 8; ++i) dst[i] = e2m1_to_float(c >> (4 * i)) * f;
    }
    __syncthreads();
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + warp * 4 + i, j = r / G;
      if (j >= n) continue;
      const float* qr = sq + (warp * 4 + i) * kHeadDim;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int d = 0; d < kHeadDim; ++d)
        for (int t = 0; t < 4; ++t) x[t] = fmaf(qr[d], sk[(lane + 32 * t) * kPitch + d], x[t]);
      bool see[4];
      float mx = m[i];
      for (int t = 0; t < 4; ++t) {
        const int64_t tok = pg * kPageTokens + lane + 32 * t;
        const int64_t pos = base + s_depth[j];
        see[t] = tok < L;
        if (tok < base) {
          see[t] &= a.window == 0 || tok > pos - a.window || tok < a.sinks;
        } else if (see[t]) {
          const int nd = (int)(tok - base);
          const int64_t at = base + s_depth[nd];
          see[t] = ((s_mask[j] >> nd) & 1) &&
                   (a.window == 0 || at > pos - a.window || at < a.sinks);
        }
        if (see[t]) mx = fmaxf(mx, x[t]);
      }
      for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
      if (mx == -INFINITY) {
        if (!__any_sync(0xFFFFFFFFu, see[0] || see[1] || see[2] || see[3])) continue;
        mx = 0.f;  // NaN logits only
      }
      const float f = expf(m[i] - mx);
      m[i] = mx;
      float ls = 0.f;
      uint32_t seen[4];
      for (int t = 0; t < 4; ++t) {
        const float p = see[t] ? expf(x[t] - mx) : 0.f;
        sp[warp * kPageTokens + lane + 32 * t] = p;
        ls += p;
        seen[t] = __ballot_sync(0xFFFFFFFFu, see[t]);
      }
      for (int d = 16; d > 0; d >>= 1) ls += __shfl_xor_sync(0xFFFFFFFFu, ls, d);
      l[i] = l[i] * f + ls;
      __syncwarp();
      for (int d = 0; d < 4; ++d) o[i][d] *= f;
      for (int t = 0; t < kPageTokens; ++t)
        if ((seen[t >> 5] >> (t & 31)) & 1u) {
          const float p = sp[warp * kPageTokens + t];
          for (int d = 0; d < 4; ++d) o[i][d] = fmaf(p, sv[t * kPitch + lane + 32 * d], o[i][d]);
        }
      __syncwarp();
    }
  }
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + warp * 4 + i, j = r / G, g = r % G;
    if (j >= a.N) continue;
    const int64_t row = (s * a.N + j) * a.H + h * G + g;
    for (int d = 0; d < 4; ++d) {
      const float v = l[i] == 0.f ? 0.f : o[i][d] / l[i];
      a.out[row * kHeadDim + lane + 32 * d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    if (lane == 0 && a.lse) a.lse[row] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
}

size_t tree_decode_workspace_bytes(int64_t, int, int, int, int) { return 0; }

cudaError_t launch_tree_decode(const uint16_t* q, int64_t B, int N, int H, int Hkv,
                               const uint8_t* k_pages, const uint8_t* v_pages, int64_t page_stride,
                               int64_t head_stride, int64_t num_pages, const int32_t* table,
                               int64_t bt_width, const int32_t* seq_lens, const int32_t* n_nodes,
                               const uint64_t* mask, int64_t window, int64_t sinks, float scale,
                               uint16_t* out, float* lse, void*, uint32_t* status, int,
                               cudaStream_t stream) {
  const TreeArgs a{q, N, H, Hkv, k_pages, v_pages, page_stride, head_stride, num_pages, table,
                   bt_width, seq_lens, n_nodes, mask, window, sinks, scale, out, lse, status};
  const size_t smem = (2 * kPageTokens * kPitch + kRows * kHeadDim + kTreeWarps * kPageTokens) * 4;
  cudaError_t e = cudaFuncSetAttribute(tree_simple_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_simple_kernel,
                    dim3((unsigned)((N * (H / Hkv) + kRows - 1) / kRows), Hkv, (unsigned)B),
                    dim3(kTreeWarps * 32), smem, stream, a);
}

}  // namespace mx4
