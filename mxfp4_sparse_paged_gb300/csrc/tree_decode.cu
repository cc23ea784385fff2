// tree_paged_decode: attention of a speculative step's nodes over the MXFP4 pages, on
// the tensor cores.
//
// A row is one (node, query head of the group) pair; a tile is NR rows of one sequence
// and KV head.  Everything is computed transposed, with the page's 128 tokens (then the
// 128 dims) on the tensor core's M side and the rows on its N side, so that a single
// token's 16 heads take an N of 16 and not an eighth of an M of 128:
//   S^T[token, row] = K q^T      tcgen05.mma kind::mxf8f6f4.block_scale, A = the page's e2m1
//                                rows and e8m0 scales as they are stored, no dequantisation;
//   P^T = 2^(scale log2e S - ref) rounded to bf16;
//   O^T[dim, row] += V^T P^T     tcgen05.mma kind::f16 on bf16.
//
// q as a sum of two E4M3 numbers.  The block-scaled product wants q in an MX format.  A bf16
// has 8 significant bits: hi = E4M3(q 2^-E) takes the first 4 (E puts the 32-block's largest
// element in [2^7, 2^8)), lo = E4M3((q 2^-E - hi) 2^5) the rest exactly, down to 2^-14 of the
// largest element and to 2^-22 of it in absolute terms.  Two MMAs into one accumulator.
//
// V.  Its scales run along the contraction's other axis, so V is dequantised into a bf16
// operand in shared memory, exactly: an e2m1 code's bits moved to a bf16's sign, low
// exponent and first mantissa bit read as the code's value times 2^-126 (e = 0 being
// bf16's subnormals), and one multiplication by 2^(s - 1) gives the value.
//
// Softmax.  bf16 and fp32 hold the weights to the same relative precision at any size, so
// the reference of a row need not be its running maximum: it is the maximum of the page
// that set it, and stays until a logit lies 2^kLazy above it.  Only then (and on the first
// page) is there a reduction over the tokens, which lie across lanes; a page otherwise
// costs one vote.  Row sums stay in the lanes until the end of the tile.
//
// Work.  The pages of all tiles, in order, are cut into equal contiguous ranges, one per
// CTA.  A tile cut by a range's end leaves a partial record (O, reference, sum) in the
// workspace, and a second kernel joins the records of each cut tile.
//
// Roles.  Warp 0 streams pages (tensor copy of K into the operand's swizzled layout, bulk
// copies of scales and of V), warp 1 issues the MMAs, warps 4-7 do the softmax (one lane a
// token; in the epilogue one lane a dim), warps 8-11 convert q and dequantise V.  All waits
// are bounded; after one that runs out every role goes through its loop without waiting or
// issuing, and the status word says so.
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled
#include <cuda_bf16.h>

#include <algorithm>

#include "score_pipeline.cuh"

namespace mx4 {

namespace tree {

constexpr int kThreads = 384;
constexpr int kMaxSeq = 512;       // sequences per launch
constexpr float kLazy = 12.f;      // log2 units a logit may lie above its row's reference
constexpr float kUnset = -3e38f;   // the reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKStage = 128 * 128 + 512;  // K operand tile, scales
constexpr int kVTile = 128 * 128 * 2;

struct Args {
  CUtensorMap tmap;  // the K pool
  const uint16_t* q;
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
  float* rec;   // [grid][2][NR * 130] partial records
  int32_t* meta;  // [grid][4]
  uint32_t* status;
  int B, N, H, Hkv, G, tiles;
};

// Shared-memory layout, in bytes.
template <int NR, int VB, int STG>
struct Lay {
  static constexpr int kK = 0;                         // [STG] K operand | scales
  static constexpr int kKPitch = (kKStage + 1023) / 1024 * 1024;
  static constexpr int kVraw = kK + STG * kKPitch;     // [STG] V pages as stored
  static constexpr int kV = kVraw + STG * kPageBytes;  // [VB] V operand
  static constexpr int kP = kV + VB * kVTile;          // [VB] P operand
  static constexpr int kQ = kP + VB * NR * 256;        // q operand: hi, lo
  static constexpr int kSf = kQ + 2 * NR * 128;        // q scale words: hi, lo
  static constexpr int kRef = kSf + 2 * NR * 4;        // [NR] references
  static constexpr int kFac = kRef + NR * 4;           // [NR] rescaling factors, then 1 / sum
  static constexpr int kWarp = kFac + NR * 4;          // [4][NR] per-warp maxima and sums
  static constexpr int kNan = kWarp + 4 * NR * 4;      // [NR] dim blocks with a visible NaN
  static constexpr int kNode = kNan + NR * 4;          // [NR] output row, -1 none
  static constexpr int kDepth = kNode + NR * 4;        // [NR]
  static constexpr int kMask = kDepth + NR * 4;        // [NR] u64: nodes that the row sees
  static constexpr int kPref = kMask + NR * 8;         // [kMaxSeq] i64 page prefix
  static constexpr int kLen = kPref + kMaxSeq * 8;     // [kMaxSeq]
  static constexpr int kCnt = kLen + kMaxSeq * 4;      // [kMaxSeq] u8
  static constexpr int kInfo = kCnt + kMaxSeq;         // [STG] valid tokens of the page
  static constexpr int kBar = (kInfo + STG * 4 + 7) / 8 * 8;
  static constexpr int kBars = 4 * STG + 4 + 3 * VB + 4;
  static constexpr int kMisc = kBar + kBars * 8;       // abort, tmem address, scan space
  static constexpr int kBytes = kMisc + 256 + 1024;    // + slack for the 1024-byte alignment
};

template <int NR>
struct Tm {  // tensor-memory columns
  static constexpr int kS = 0;                    // two S buffers
  static constexpr int kO = 2 * NR;
  static constexpr int kSfa = 3 * NR;             // two sets of 4
  static constexpr int kSfb = kSfa + 8;           // hi, lo
  static constexpr int kSfbW = (NR + 31) / 32;    // columns of each, in a field of 4
  static constexpr int kSfbPitch = 4;             // (scale fields start at multiples of 4)
  static_assert(kSfbW <= kSfbPitch && kSfa % 4 == 0 && kSfb % 4 == 0, "scale fields");
  static constexpr int kUsed = kSfb + 2 * kSfbPitch;
  static constexpr int kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
};

__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}
// S^T: A e2m1, B e4m3, UE8M0 scales, M = 128, scale byte kb of both words
template <int NR>
__device__ constexpr uint32_t idesc_s(uint32_t kb) {
  return (kb << 4) | (5u << 7) | ((uint32_t)(NR >> 3) << 17) | (1u << 23) | (8u << 24) | (kb << 29);
}
// O^T: bf16 operands, fp32 accumulator, both with the M (N) axis contiguous
template <int NR>
__device__ constexpr uint32_t idesc_o() {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
         ((uint32_t)(NR >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 16 columns of this warp's lane quarter.
__device__ __forceinline__ void ld16(uint32_t taddr, float* x) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void st16(uint32_t taddr, const float* x) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16_mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Column sums (maxima) over a warp's lanes of 16 values a lane: lane l returns column
// l % 16's.  Each step halves the columns a lane holds: 16 shuffles, not 80.
template <class Op>
__device__ __forceinline__ float columns16(const float* in, int lane, Op op) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = in[i];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
    }
  }
  return op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 16));
}

// What a sequence's cached tokens give its tiles: pages 0 .. ns-1 hold the first
// `sinks` tokens, pages first .. the window and the drafts.
struct Span {
  int64_t base;  // tokens before the drafts
  int len, n, ns, first, np;
};
__device__ __forceinline__ Span span_of(int64_t L, int n, int64_t window, int64_t sinks) {
  Span sp;
  sp.len = (int)L;
  sp.n = n;
  sp.base = L - n;
  const int64_t lo = window > 0 ? max((int64_t)0, sp.base + 1 - window) : 0;
  sp.first = (int)(lo / kPageTokens);
  sp.ns = (int)min((min(sinks, lo) + kPageTokens - 1) / kPageTokens, (int64_t)sp.first);
  sp.np = n > 0 ? sp.ns + (int)((L + kPageTokens - 1) / kPageTokens) - sp.first : 0;
  return sp;
}

__host__ __device__ __forceinline__ int64_t range_begin(int64_t g, int64_t U, int64_t G) {
  return U * g / G;
}

template <int NR, int VB, int STG, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) kernel(const __grid_constant__ Args a) {
  using L_ = Lay<NR, VB, STG>;
  using T_ = Tm<NR>;
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t* const s_pref = reinterpret_cast<int64_t*>(sm + L_::kPref);
  int* const s_len = reinterpret_cast<int*>(sm + L_::kLen);
  uint8_t* const s_cnt = sm + L_::kCnt;
  volatile int* const s_info = reinterpret_cast<volatile int*>(sm + L_::kInfo);
  volatile int* const s_abort = reinterpret_cast<volatile int*>(sm + L_::kMisc);
  uint32_t* const s_taddr = reinterpret_cast<uint32_t*>(sm + L_::kMisc + 4);
  int64_t* const s_scan = reinterpret_cast<int64_t*>(sm + L_::kMisc + 16);  // [12]
  auto bar = [&](int i) { return sb + L_::kBar + 8u * i; };
  const int kKFull = 0, kKEmpty = STG, kVFull = 2 * STG, kVEmpty = 3 * STG, kSFull = 4 * STG,
            kSFree = kSFull + 2, kPFull = kSFree + 2, kVReady = kPFull + VB, kPvDone = kVReady + VB,
            kQFull = kPvDone + VB, kQEmpty = kQFull + 1, kOFree = kQEmpty + 1, kDrain = kOFree + 1;

  if (tid == 0) {
    for (int i = 0; i < STG; ++i) {
      mbar_init(bar(kKFull + i), 1);
      mbar_init(bar(kKEmpty + i), 1);
      mbar_init(bar(kVFull + i), 1);
      mbar_init(bar(kVEmpty + i), 8);  // four dequantising warps, four softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kSFree + i), 4);
    }
    for (int i = 0; i < VB; ++i) {
      mbar_init(bar(kPFull + i), 4);
      mbar_init(bar(kVReady + i), 4);
      mbar_init(bar(kPvDone + i), 1);
    }
    mbar_init(bar(kQFull), 4);
    mbar_init(bar(kQEmpty), 1);
    mbar_init(bar(kOFree), 4);
    mbar_init(bar(kDrain), 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  // The kernel in front may hold tensor memory that this one would wait for: its end first.
  pdl_wait();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_addr(s_taddr)),
                 "r"(T_::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  // ---- pages a sequence and their prefix sum (a tile without pages counts as one)
  {
    constexpr int per = (kMaxSeq + kThreads - 1) / kThreads;
    int64_t mine[per], sum = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      mine[i] = 0;
      if (s < a.B) {
        int64_t L = a.seq_lens[s];
        int n = a.n_nodes ? a.n_nodes[s] : a.N;
        if (n < 0 || n > a.N || L < n || L > a.bt_width * kPageTokens) {
          if (blockIdx.x == 0) flag(a.status, MX4_STATUS_BAD_LEN);
          n = 0;
          L = 0;
        }
        s_len[s] = (int)L;
        s_cnt[s] = (uint8_t)n;
        mine[i] = max(1, span_of(L, n, a.window, a.sinks).np);
      }
      sum += mine[i];
    }
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
    for (int w = 0; w < warp; ++w) before += s_scan[w];
#pragma unroll
    for (int i = 0; i < per; ++i) {
      before += mine[i];
      if (tid * per + i < a.B) s_pref[tid * per + i] = before;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_launch_dependents();  // after this CTA has its tensor memory

  const uint32_t tm = *s_taddr;
  const int HT = a.Hkv * a.tiles;
  const int64_t U = s_pref[a.B - 1] * HT;
  // few pages a CTA are not worth the records: at least kMinPages each
  constexpr int kMinPages = 2;
  const int64_t Gd = max((int64_t)1, min((int64_t)gridDim.x, U / kMinPages));
  const int64_t g = blockIdx.x;
  const int64_t u0 = g < Gd ? range_begin(g, U, Gd) : U, u1 = g < Gd ? range_begin(g + 1, U, Gd) : U;

  auto wait = [&](int i, uint32_t parity) -> bool {
    const uint32_t b = bar(i);
    for (uint32_t p = 0; p < kWaitPolls; ++p) {
      if (mbar_test(b, parity)) return true;
      if ((p & 63u) == 63u && *s_abort) return false;
    }
    *s_abort = 1;
    flag(a.status, MX4_STATUS_TIMEOUT);
    return false;
  };

  // The tiles of this CTA's range, in order: f(tile number in the range, sequence, head,
  // row tile, its span, its pages [e0, e1) of this range, begins, ends).
  auto for_tiles = [&](auto&& f) {
    int64_t u = u0;
    int s = 0, ht = 0, count = 0;
    int64_t e = 0;
    if (u < u1) {
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] * HT > u) hi = mid; else lo = mid + 1;
      }
      s = lo;
      const int64_t p0 = s > 0 ? s_pref[s - 1] : 0, np = s_pref[s] - p0, r = u - p0 * HT;
      ht = (int)(r / np);
      e = r - ht * np;
    }
    while (u < u1) {
      const int64_t np = s_pref[s] - (s > 0 ? s_pref[s - 1] : 0);
      const int64_t e1 = min(np, e + (u1 - u));
      const Span sp = span_of(s_len[s], s_cnt[s], a.window, a.sinks);
      f(count, s, ht / a.tiles, ht % a.tiles, sp, (int)e, (int)e1, e == 0, e1 == np);
      count += sp.np > 0;
      u += e1 - e;
      e = 0;
      if (++ht == HT) {
        ht = 0;
        ++s;
      }
    }
  };
  auto page_no = [](const Span& sp, int e) { return e < sp.ns ? e : sp.first + (e - sp.ns); };

  if (warp == 0) {
    // ================= producer: one lane
    if (lane == 0) {
      int k = 0;
      for_tiles([&](int, int s, int h, int, const Span& sp, int e0, int e1, bool, bool) {
        if (sp.np == 0) return;
        for (int e = e0; e < e1; ++e, ++k) {
          const int pg = page_no(sp, e), st = k % STG, round = k / STG;
          const int32_t pid = a.table[(int64_t)s * a.bt_width + pg];
          const bool ok = pid >= 0 && pid < a.num_pages;
          if (!ok) flag(a.status, MX4_STATUS_BAD_PAGE);
          bool go = !*s_abort;
          if (round > 0) go = wait(kKEmpty + st, (round - 1) & 1) && go;
          if (round > 0) go = wait(kVEmpty + st, (round - 1) & 1) && go;
          if (!go) continue;
          s_info[st] = ok ? min(kPageTokens, sp.len - pg * kPageTokens) : 0;
          if (ok) {
            const uint32_t kd = sb + L_::kK + st * L_::kKPitch, vd = sb + L_::kVraw + st * kPageBytes;
            const int64_t off = (int64_t)pid * a.page_stride + (int64_t)h * a.head_stride;
            mbar_arrive_expect_tx(bar(kKFull + st), kRowDataBytes * kPageTokens + 512);
            asm volatile(
                "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::"r"(kd),
                "l"(reinterpret_cast<uint64_t>(&a.tmap)), "r"(0), "r"(0), "r"(0), "r"(h), "r"(pid),
                "r"(bar(kKFull + st))
                : "memory");
            bulk_copy_g2s(kd + 128 * 128, a.k_pages + off + kScaleOffset, 512, bar(kKFull + st));
            mbar_arrive_expect_tx(bar(kVFull + st), kPageBytes);
            bulk_copy_g2s(vd, a.v_pages + off, kPageBytes, bar(kVFull + st));
          } else {
            mbar_arrive(bar(kKFull + st));
            mbar_arrive(bar(kVFull + st));
          }
        }
      });
      // every copy has landed before the CTA ends
      for (int i = max(0, k - STG); i < k; ++i) {
        wait(kKFull + i % STG, (i / STG) & 1);
        wait(kVFull + i % STG, (i / STG) & 1);
      }
    }
  } else if (warp == 1) {
    // ================= MMA issue: one lane
    if (lane == 0) {
      int k = 0;
      bool any = false;
      // the page whose P V product is still to be issued
      int pv = -1;
      bool pv_first = false;
      int pv_tile = 0;
      auto issue_pv = [&]() {
        const int b = pv % VB;
        bool go = wait(kPFull + b, (pv / VB) & 1);
        go = wait(kVReady + b, (pv / VB) & 1) && go;
        if (pv_first && pv_tile > 0) go = wait(kOFree, (pv_tile - 1) & 1) && go;
        if (!go || *s_abort) return;
        fence_after();
        const uint32_t va = sb + L_::kV + b * kVTile, pa = sb + L_::kP + b * NR * 256;
#pragma unroll
        for (uint32_t ks = 0; ks < 8; ++ks) {
          const uint64_t ad = desc(va + ks * 256, 128, 2048), bd = desc(pa + ks * 256, 128, 2048);
          asm volatile(
              "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
              " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tm + T_::kO),
              "l"(ad), "l"(bd), "r"(idesc_o<NR>()), "r"((uint32_t)(ks > 0 || !pv_first))
              : "memory");
        }
        commit(bar(kPvDone + b));
      };
      for_tiles([&](int tile, int, int, int, const Span& sp, int e0, int e1, bool, bool) {
        if (sp.np == 0) return;
        any = true;
        for (int e = e0; e < e1; ++e, ++k) {
          const int st = k % STG, b = k & 1;
          bool go = true;
          if (e == e0) go = wait(kQFull, tile & 1);
          go = wait(kKFull + st, (k / STG) & 1) && go;
          if (k >= 2) go = wait(kSFree + b, ((k >> 1) - 1) & 1) && go;
          if (go && !*s_abort) {
            fence_after();
            const uint32_t ka = sb + L_::kK + st * L_::kKPitch, qa = sb + L_::kQ;
            const uint32_t sfa = tm + T_::kSfa + 4u * b;
            asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(sfa),
                         "l"(desc(ka + 128 * 128, 16, 128))
                         : "memory");
#pragma unroll
            for (uint32_t part = 0; part < 2; ++part)
#pragma unroll
              for (uint32_t kb = 0; kb < 4; ++kb) {
                const uint64_t ad = desc(ka + kb * 32, 16, 1024) | ((uint64_t)2 << 61);
                const uint64_t bd = desc(qa + part * NR * 128 + kb * 256, 128, 1024);
                asm volatile(
                    "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                    " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, "
                    "%2, %3, [%4], [%5], p;\n}\n" ::"r"(tm + T_::kS + b * NR),
                    "l"(ad), "l"(bd), "r"(idesc_s<NR>(kb)), "r"(sfa),
                    "r"(tm + T_::kSfb + part * T_::kSfbPitch), "r"(part + kb)
                    : "memory");
              }
            commit(bar(kSFull + b));
            commit(bar(kKEmpty + st));
            if (e == e1 - 1) commit(bar(kQEmpty));
          }
          if (pv >= 0) issue_pv();
          pv = k;
          pv_first = e == e0;
          pv_tile = tile;
        }
      });
      if (pv >= 0) issue_pv();
      if (any) {  // no MMA in flight when the tensor memory is freed
        commit(bar(kDrain));
        for (uint32_t p = 0; p < kWaitPolls; ++p)
          if (mbar_test(bar(kDrain), 0)) break;
      }
    }
  } else if (warp >= 8) {
    // ================= q conversion and V dequantisation
    const int t = tid - 256, w = warp - 8;
    const int r8 = lane & 7, blk = ((r8 >> 1) + (lane >> 3)) & 3;  // see below
    int k = 0;
    for_tiles([&](int tile, int s, int h, int rt, const Span& sp, int e0, int e1, bool, bool) {
      if (sp.np == 0) return;
      if (tile > 0) wait(kQEmpty, (tile - 1) & 1);
      // 16 elements a thread: K-chunk j of row n; the two threads of a 32-block share its
      // largest magnitude
      for (int n = t >> 3; n < NR; n += 16) {
        const int j = t & 7, row = rt * NR + n, node = row / a.G;
        uint32_t wd[8] = {};
        float amax = 0.f;
        if (node < sp.n) {
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (((int64_t)s * a.N + node) * a.H + h * a.G + row % a.G) * kHeadDim + 16 * j);
          const uint4 x0 = src[0], x1 = src[1];
          wd[0] = x0.x; wd[1] = x0.y; wd[2] = x0.z; wd[3] = x0.w;
          wd[4] = x1.x; wd[5] = x1.y; wd[6] = x1.z; wd[7] = x1.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_float(wd[i] & 0xFFFFu)),
                                   fabsf(bf16_bits_to_float(wd[i] >> 16))));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        const int ef = min(254, (int)(__float_as_uint(amax) >> 23));
        const int E = amax == 0.f ? 0 : max(-122, ef - 127 - 7);
        const float inv = __uint_as_float((uint32_t)(127 - E) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t hc[2], lc[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x2 = wd[2 * i + u];
            float x0 = bf16_bits_to_float(x2 & 0xFFFFu), x1 = bf16_bits_to_float(x2 >> 16);
            // an infinity has no E4M3 code: NaN, as its logits would be
            x0 = isinf(x0) ? NAN : x0 * inv;
            x1 = isinf(x1) ? NAN : x1 * inv;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n" : "=h"(hc[u]) : "f"(x0), "f"(x1));
            uint32_t hf;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(hf) : "h"(hc[u]));
            const float h0 = __half2float(__ushort_as_half((unsigned short)(hf & 0xFFFFu)));
            const float h1 = __half2float(__ushort_as_half((unsigned short)(hf >> 16)));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n"
                : "=h"(lc[u])
                : "f"((x0 - h0) * 32.f), "f"((x1 - h1) * 32.f));
          }
          hi[i] = (uint32_t)hc[0] | ((uint32_t)hc[1] << 16);
          lo[i] = (uint32_t)lc[0] | ((uint32_t)lc[1] << 16);
        }
        uint8_t* dst = sm + L_::kQ + (n >> 3) * 1024 + j * 128 + (n & 7) * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + NR * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if ((j & 1) == 0) {
          sm[L_::kSf + n * 4 + (j >> 1)] = (uint8_t)(E + 127);
          sm[L_::kSf + (NR + n) * 4 + (j >> 1)] = (uint8_t)(E + 122);
        }
      }
      fence_async();
      asm volatile("bar.sync 2, 128;\n" ::: "memory");
      // row n's scale word at lane n % 32 of every lane quarter, column n / 32
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int c = 0; c < T_::kSfbW; ++c)
          st1(tm + ((uint32_t)(32 * w) << 16) + T_::kSfb + part * T_::kSfbPitch + c,
              *reinterpret_cast<const uint32_t*>(
                  sm + L_::kSf + (part * NR + min(NR - 1, c * 32 + lane)) * 4));
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));

      for (int e = e0; e < e1; ++e, ++k) {
        const int st = k % STG, b = k % VB;
        wait(kVFull + st, (k / STG) & 1);
        if (k >= VB) wait(kPvDone + b, (k / VB - 1) & 1);
        const int live = s_info[st];
        const uint8_t* raw = sm + L_::kVraw + st * kPageBytes;
        uint8_t* const vb = sm + L_::kV + b * kVTile;
        // Operand row (K index) m holds token 4 (m % 32) + m / 32, the order in which the
        // tensor copy lays out K.  A warp's step: the 8 operand rows of one core matrix
        // (r8), lane >> 3 choosing which 32-dim block of each: 16 raw bytes a lane, four
        // 16-byte stores without bank conflicts.
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int m = (w * 4 + it) * 8 + r8;
          const int tok = 4 * (m & 31) + (m >> 5);
          const uint4 c4 = *reinterpret_cast<const uint4*>(raw + tok * kRowDataBytes + blk * 16);
          const uint32_t sc = raw[kScaleOffset + tok * kRowScaleBytes + blk];
          const bool use = tok < live && sc != 255u;
          // 2^(sc - 1), as two factors where it passes bf16's range
          const uint32_t e1x = use ? min(sc + 126u, 254u) : 0u;
          const uint32_t f1 = (e1x << 7) * 0x10001u;
          const uint32_t f2 = ((127u + (sc > 128u ? sc - 128u : 0u)) << 7) * 0x10001u;
          const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t x = cw[j];
            // codes i and i + 4 of the word as one pair
            uint32_t y[4];
            y[0] = ((x << 12) & 0x80008000u) | ((x << 6) & 0x01C001C0u);
            y[1] = ((x << 8) & 0x80008000u) | ((x << 2) & 0x01C001C0u);
            y[2] = ((x << 4) & 0x80008000u) | ((x >> 2) & 0x01C001C0u);
            y[3] = (x & 0x80008000u) | ((x >> 6) & 0x01C001C0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = bf16_mul2(y[i], f1);
            if (sc > 128u)
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = bf16_mul2(y[i], f2);
            *reinterpret_cast<uint4*>(vb + (blk * 4 + j) * 2048 + (m >> 3) * 128 + r8 * 16) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kVReady + b));
          mbar_arrive(bar(kVEmpty + st));
        }
      }
    });
  } else if (warp >= 4) {
    // ================= softmax
    const int t = tid - 128, w = warp - 4;
    const uint32_t tl = tm + ((uint32_t)(32 * w) << 16);
    float* const s_ref = reinterpret_cast<float*>(sm + L_::kRef);
    float* const s_fac = reinterpret_cast<float*>(sm + L_::kFac);
    float* const s_warp = reinterpret_cast<float*>(sm + L_::kWarp);
    uint32_t* const s_nan = reinterpret_cast<uint32_t*>(sm + L_::kNan);
    int* const s_node = reinterpret_cast<int*>(sm + L_::kNode);
    int* const s_depth = reinterpret_cast<int*>(sm + L_::kDepth);
    uint64_t* const s_mask = reinterpret_cast<uint64_t*>(sm + L_::kMask);
    auto sync4 = []() { asm volatile("bar.sync 1, 128;\n" ::: "memory"); };
    auto any4 = [](bool v) {
      uint32_t r;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
          " barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(r)
          : "r"((uint32_t)v)
          : "memory");
      return r != 0u;
    };
    const float cs = a.scale * kLog2e;
    const int tok = 4 * lane + w;  // this lane's token of a page
    int k = 0;
    for_tiles([&](int tile, int s, int h, int rt, const Span& sp, int e0, int e1, bool begins,
                  bool ends) {
      // ---- the tile's rows
      sync4();  // the tile before is written out
      for (int c = t; c < NR; c += 128) {
        const int row = rt * NR + c, node = row / a.G;
        s_node[c] = node < a.N ? node * a.H + h * a.G + row % a.G : -1;
        uint64_t mk = 0;
        int d = 0;
        if (node < sp.n) {
          const uint64_t all = sp.n < 64 ? (1ull << sp.n) - 1 : ~0ull;
          auto mask_of = [&](int j) {
            return (a.mask ? a.mask[(int64_t)s * a.N + j] : (2ull << j) - 1) & all;
          };
          auto depth_of = [&](int j) { return max(1, __popcll(mask_of(j))) - 1; };
          mk = mask_of(node);
          d = depth_of(node);
          if (a.window > 0)
            for (int i = 0; i < sp.n; ++i)
              if ((mk >> i) & 1ull) {
                const int di = depth_of(i);
                if (!(di > d - a.window || sp.base + di < a.sinks)) mk &= ~(1ull << i);
              }
        } else {
          d = -1;  // no node: sees nothing, whatever is computed for it
        }
        s_mask[c] = mk;
        s_depth[c] = d;
        s_ref[c] = kUnset;
        s_nan[c] = 0;
      }
      sync4();
      float l[NR];
#pragma unroll
      for (int c = 0; c < NR; ++c) l[c] = 0.f;

      if (sp.np > 0) {
        for (int e = e0; e < e1; ++e, ++k) {
          const int st = k % STG, b = k & 1, pb = k % VB;
          const int64_t first = (int64_t)page_no(sp, e) * kPageTokens, i_g = first + tok;
          wait(kVFull + st, (k / STG) & 1);
          const int live = s_info[st];
          uint32_t vw = *reinterpret_cast<const uint32_t*>(sm + L_::kVraw + st * kPageBytes +
                                                           kScaleOffset + tok * kRowScaleBytes);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kVEmpty + st));
          // dim blocks of this token's V row that are NaN
          vw = ((vw & 0x7F7F7F7Fu) + 0x01010101u) & vw & 0x80808080u;
          const bool plain = live == kPageTokens && first + kPageTokens <= sp.base &&
                             (a.window == 0 || first > sp.base + 63 - a.window ||
                              first + kPageTokens <= a.sinks);
          auto sees = [&](int c) {
            if (tok >= live || s_depth[c] < 0) return false;
            if (i_g >= sp.base) return ((s_mask[c] >> (int)(i_g - sp.base)) & 1ull) != 0;
            return a.window == 0 || i_g > sp.base + s_depth[c] - a.window || i_g < a.sinks;
          };
          wait(kSFull + b, (k >> 1) & 1);
          fence_after();
          float x[NR];
          auto logits = [&]() {
#pragma unroll
            for (int c = 0; c < NR; c += 16) ld16(tl + T_::kS + b * NR + c, x + c);
            wait_ld();
          };
          auto hide = [&]() {  // -inf where not seen, whatever was computed there
            if (!plain) {
#pragma unroll
              for (int c = 0; c < NR; ++c)
                if (!sees(c)) x[c] = -INFINITY;
            }
          };
          logits();
#pragma unroll
          for (int c = 0; c < NR; c += 4) {
            const float4 rf = *reinterpret_cast<const float4*>(s_ref + c);
            x[c] = fmaf(x[c], cs, -rf.x);
            x[c + 1] = fmaf(x[c + 1], cs, -rf.y);
            x[c + 2] = fmaf(x[c + 2], cs, -rf.z);
            x[c + 3] = fmaf(x[c + 3], cs, -rf.w);
          }
          hide();
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < NR; ++c) top = fmaxf(top, x[c]);
          if (any4(top > kLazy)) {
            // new references: the page's maximum of each row that has a larger one
            logits();
#pragma unroll
            for (int c = 0; c < NR; ++c) x[c] = x[c] * cs;
            hide();
#pragma unroll
            for (int c = 0; c < NR; c += 16) {
              const float v = columns16(x + c, lane, [](float p, float q) { return fmaxf(p, q); });
              if (lane < 16) s_warp[w * NR + c + lane] = v;
            }
            if (k > 0 && e > e0) wait(kPvDone + (k - 1) % VB, ((k - 1) / VB) & 1);
            sync4();
            for (int c = t; c < NR; c += 128) {
              const float v = fmaxf(fmaxf(s_warp[c], s_warp[NR + c]),
                                    fmaxf(s_warp[2 * NR + c], s_warp[3 * NR + c]));
              const float old = s_ref[c], now = fmaxf(old, v);
              s_fac[c] = old == kUnset ? 0.f : ex2(old - now);
              s_ref[c] = now;
            }
            sync4();
#pragma unroll
            for (int c = 0; c < NR; ++c) {
              l[c] *= s_fac[c];
              x[c] -= s_ref[c];
            }
            if (e > e0) {
              fence_after();
#pragma unroll
              for (int c = 0; c < NR; c += 16) {
                float o[16];
                ld16(tl + T_::kO + c, o);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= s_fac[c + i];
                st16(tl + T_::kO + c, o);
              }
              wait_st();
            }
          }
          // the accumulator has been read: the next page's product may go into it
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSFree + b));
          if (vw != 0u) {
            for (int c = 0; c < NR; ++c)
              if (sees(c)) atomicOr(s_nan + c, vw);
          }
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            x[c] = ex2(x[c]);
            l[c] += x[c];
          }
          if (k >= VB) wait(kPvDone + pb, (k / VB - 1) & 1);
          uint8_t* const pd = sm + L_::kP + pb * NR * 256 + (4 * w + (lane >> 3)) * 128 + (lane & 7) * 16;
#pragma unroll
          for (int c = 0; c < NR; c += 8)
            *reinterpret_cast<uint4*>(pd + (c >> 3) * 2048) =
                make_uint4(pack_bf16(x[c], x[c + 1]), pack_bf16(x[c + 2], x[c + 3]),
                           pack_bf16(x[c + 4], x[c + 5]), pack_bf16(x[c + 6], x[c + 7]));
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kPFull + pb));
        }
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
          const float v = columns16(l + c, lane, [](float p, float q) { return p + q; });
          if (lane < 16) s_warp[w * NR + c + lane] = v;
        }
        wait(kPvDone + (k - 1) % VB, ((k - 1) / VB) & 1);
        sync4();
      } else {
        for (int c = t; c < 4 * NR; c += 128) s_warp[c] = 0.f;
        sync4();
      }
      // ---- the tile's result: this lane's dim of every row
      const bool whole = begins && ends;
      float* const rec = a.rec + (2 * g + (begins ? 1 : 0)) * (int64_t)(NR * 130);
      for (int c = t; c < NR; c += 128) {
        float sum = (s_warp[c] + s_warp[NR + c]) + (s_warp[2 * NR + c] + s_warp[3 * NR + c]);
        if (s_depth[c] < 0) sum = 0.f;
        const float rf = s_ref[c];
        if (whole) {
          s_fac[c] = sum == 0.f ? 0.f : 1.f / sum;
          if (a.lse && s_node[c] >= 0)
            a.lse[(int64_t)s * a.N * a.H + s_node[c]] =
                sum == 0.f ? -INFINITY : (log2f(sum) + (rf == kUnset ? 0.f : rf)) * 0.6931471805599453f;
        } else {
          s_fac[c] = sum == 0.f ? 0.f : 1.f;
          rec[NR * 128 + c] = rf;
          rec[NR * 129 + c] = sum;
        }
      }
      sync4();
      fence_after();
      // operand position -> dim: the codes of a word were paired i, i + 4
      const int dim = 32 * w + (lane & 24) + ((lane & 1) << 2) + ((lane & 7) >> 1);
      const uint32_t nb = 0x80u << (8 * w);
      for (int c = 0; c < NR; c += 16) {
        float o[16];
        if (sp.np > 0) {
          ld16(tl + T_::kO + c, o);
          wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float f = s_fac[c + i];
          float v = f == 0.f ? 0.f : o[i] * f;
          if (s_nan[c + i] & nb) v = NAN;
          if (whole) {
            const int nd = s_node[c + i];
            if (nd >= 0)
              a.out[((int64_t)s * a.N * a.H + nd) * kHeadDim + dim] =
                  __bfloat16_as_ushort(__float2bfloat16_rn(v));
          } else {
            rec[(c + i) * 128 + dim] = v;
          }
        }
      }
      fence_before();
      __syncwarp();
      if (sp.np > 0 && lane == 0) mbar_arrive(bar(kOFree));
      // a tile that began in a range before this one: if that range's end is the tile's
      // first cut, this CTA's place in the list says how many records join
      if (t == 0 && !begins && e0 > 0) {
        const int64_t start = u0 - e0, end = start + max(1, sp.np);
        if (range_begin(g - 1, U, Gd) <= start) {
          int parts = 2;
          while (g + parts - 1 < Gd && range_begin(g + parts - 1, U, Gd) < end) ++parts;
          a.meta[4 * g + 1] = s;
          a.meta[4 * g + 2] = h * a.tiles + rt;
          a.meta[4 * g] = parts;
        } else {
          a.meta[4 * g] = 0;
        }
      }
    });
    // no cut tile at this range's start
    if (t == 0) {
      bool cut = false;
      if (u0 < u1) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_pref[mid] * HT > u0) hi = mid; else lo = mid + 1;
        }
        const int64_t p0 = lo > 0 ? s_pref[lo - 1] : 0;
        cut = (u0 - p0 * HT) % (s_pref[lo] - p0) != 0;
      }
      if (!cut) a.meta[4 * g] = 0;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tm), "r"(T_::kCols)
                 : "memory");
}

// Joins the records of a cut tile: block x = the range after its first cut, a warp a row,
// a lane four dims: out = sum_r O_r 2^(m_r - M) / sum_r l_r 2^(m_r - M).
template <int NR>
__global__ void __launch_bounds__(128) merge_kernel(const Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t g = blockIdx.x;
  const int parts = a.meta[4 * g];
  if (parts < 2) return;
  const int s = a.meta[4 * g + 1], ht = a.meta[4 * g + 2];
  const int h = ht / a.tiles, rt = ht % a.tiles, lane = threadIdx.x & 31;
  const int c = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int row = rt * NR + c, node = row / a.G;
  if (node >= a.N) return;
  // the first record is the last of range g - 1, the others the first of theirs
  auto rec = [&](int p) {
    return a.rec + (p == 0 ? 2 * (g - 1) + 1 : 2 * (g - 1 + p)) * (int64_t)(NR * 130);
  };
  float M = kUnset;
  for (int p = lane; p < parts; p += 32) M = fmaxf(M, rec(p)[NR * 128 + c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float* r = rec(p);
    const float m = r[NR * 128 + c], l = r[NR * 129 + c];
    const float4 v = reinterpret_cast<const float4*>(r + c * 128)[lane];
    const float f = m == kUnset ? (l == 0.f ? 0.f : 1.f) : ex2(m - M);
    sum = fmaf(l, f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  const int64_t o = ((int64_t)s * a.N + node) * a.H + h * a.G + row % a.G;
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  uint2 y;
  y.x = pack_bf16(f == 0.f ? 0.f : acc.x * f, f == 0.f ? 0.f : acc.y * f);
  y.y = pack_bf16(f == 0.f ? 0.f : acc.z * f, f == 0.f ? 0.f : acc.w * f);
  reinterpret_cast<uint2*>(a.out + o * kHeadDim)[lane] = y;
  if (a.lse && lane == 0)
    a.lse[o] = sum == 0.f ? -INFINITY
                          : (log2f(sum) + (M == kUnset ? 0.f : M)) * 0.6931471805599453f;
}

// The K pool as a 5-d tensor: 128 4-bit elements, rows 4r + c of a page as r (32) and c
// (4), heads, pages.  A box is one page with c outermost, so operand row 32 c + r is
// token 4 r + c, and the page's scale words lie in shared memory just as the copy into
// tensor memory wants them: the words of operand rows r, 32 + r, 64 + r, 96 + r together.
static cudaError_t encode_pool(const uint8_t* pages, int64_t page_stride, int64_t head_stride,
                               int64_t num_pages, int Hkv, CUtensorMap* tm) {
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
  const cuuint64_t dims[5] = {2 * kRowDataBytes, 32, 4, (cuuint64_t)Hkv, (cuuint64_t)num_pages};
  const cuuint64_t strides[4] = {4 * kRowDataBytes, kRowDataBytes,
                                 (cuuint64_t)(Hkv > 1 ? head_stride : kPageBytes),
                                 (cuuint64_t)page_stride};
  const cuuint32_t box[5] = {2 * kRowDataBytes, 32, 4, 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 5, const_cast<uint8_t*>(pages),
                         dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int NR, int VB, int STG, int CTAS>
cudaError_t launch(Args a, int64_t B, int num_sms, cudaStream_t stream) {
  const int smem = Lay<NR, VB, STG>::kBytes;
  auto kern = kernel<NR, VB, STG, CTAS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = num_sms * CTAS;
  a.tiles = (a.N * a.G + NR - 1) / NR;
  a.meta = reinterpret_cast<int32_t*>(a.rec + (int64_t)grid * 2 * NR * 130);
  const Args all = a;
  for (int64_t b0 = 0; b0 < B; b0 += kMaxSeq) {
    a = all;
    a.B = (int)std::min<int64_t>(kMaxSeq, B - b0);
    a.q += b0 * a.N * a.H * kHeadDim;
    a.out += b0 * a.N * a.H * kHeadDim;
    if (a.lse) a.lse += b0 * a.N * a.H;
    a.table += b0 * a.bt_width;
    a.seq_lens += b0;
    if (a.n_nodes) a.n_nodes += b0;
    if (a.mask) a.mask += b0 * a.N;
    e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(merge_kernel<NR>, dim3(grid, NR / 4), dim3(128), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Rows a tile: the smallest that holds all of a sequence's rows of one KV head, else the
// largest.
inline int rows_of(int N, int H, int Hkv) {
  const int rows = N * (H / Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}
inline int ctas_of(int nr) { return nr <= 32 ? 2 : 1; }

}  // namespace tree

size_t tree_decode_workspace_bytes(int64_t, int N, int H, int Hkv, int num_sms) {
  const int nr = tree::rows_of(N, H, Hkv);
  return (size_t)num_sms * tree::ctas_of(nr) * (2 * nr * 130 * 4 + 16);
}

cudaError_t launch_tree_decode(const uint16_t* q, int64_t B, int N, int H, int Hkv,
                               const uint8_t* k_pages, const uint8_t* v_pages, int64_t page_stride,
                               int64_t head_stride, int64_t num_pages, const int32_t* table,
                               int64_t bt_width, const int32_t* seq_lens, const int32_t* n_nodes,
                               const uint64_t* mask, int64_t window, int64_t sinks, float scale,
                               uint16_t* out, float* lse, void* ws, uint32_t* status, int num_sms,
                               cudaStream_t stream) {
  tree::Args a;
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.page_stride = page_stride;
  a.head_stride = head_stride;
  a.num_pages = num_pages;
  a.table = table;
  a.bt_width = bt_width;
  a.seq_lens = seq_lens;
  a.n_nodes = n_nodes;
  a.mask = mask;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.rec = static_cast<float*>(ws);
  a.meta = nullptr;
  a.status = status;
  a.B = 0;
  a.N = N;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.tiles = 0;
  if (cudaError_t e = tree::encode_pool(k_pages, page_stride, head_stride, num_pages, Hkv, &a.tmap))
    return e;
  switch (tree::rows_of(N, H, Hkv)) {
    case 16: return tree::launch<16, 1, 2, 2>(a, B, num_sms, stream);
    case 32: return tree::launch<32, 1, 2, 2>(a, B, num_sms, stream);
    default: return tree::launch<64, 2, 2, 1>(a, B, num_sms, stream);
  }
}

}  // namespace mx4
