// tree_paged_decode: attention of a speculative step's nodes over the MXFP4 pages, on
// the tensor cores.
//
// A row is one (node, query head of the group) pair; a tile is NR rows of one sequence
// and KV head.  Everything is computed transposed, with the page's 128 tokens (then the
// 128 dims) on the tensor core's M side and the rows on its N side, so that a single
// token's 16 heads take an N of 16 and not an eighth of an M of 128:
//   S^T[token, row] = K q^T      tcgen05.mma kind::mxf8f6f4.block_scale, A = the page's e2m1
//                                rows and e8m0 scales as they are stored, no dequantisation;
//   P^T = 2^(scale log2e (S - ref)) rounded to bf16;
//   O^T[dim, row] += V^T P^T     tcgen05.mma kind::f16 on bf16 (V / 4, see below).
//
// q as a sum of two E4M3 numbers.  The block-scaled product wants q in an MX format.  A bf16
// has 8 significant bits: hi = E4M3(q 2^-E) takes the first 4 (E puts the 32-block's largest
// element in [2^7, 2^8)), lo = E4M3((q 2^-E - hi) 2^5) the rest exactly, down to 2^-14 of the
// largest element and to 2^-22 of it in absolute terms.  Two MMAs into one accumulator.
//
// V.  Its scales run along the contraction's other axis, so a quarter of V is dequantised into a
// bf16 operand in shared memory, exactly: an e2m1 code's bits moved to a bf16's sign, low
// exponent and first mantissa bit read as the code's value times 2^-126 (e = 0 being
// bf16's subnormals), and one multiplication by 2^(s - 3) gives a quarter of the value; the
// results are multiplied by 4.  The largest value, 6 x 2^127, is past bf16's range: as an
// infinity it would be NaN times the weight 0 of a row that does not see it.  Its quarter is
// not, and the smallest quarter, 2^-130, is a bf16 as well.
//
// P in bf16, like the results: half a step, 2^-9, of each weight (its fp32 value goes into the row's
// sum), which takes the 2-norm error of the results from 1.7e-3, bf16's own, to 2.3e-3, and to
// 3.2e-3 where single tokens hold most of a row.  P as the sum of two bf16 numbers leaves 1.7e-3,
// but costs 256 ragged single tokens 11 % more time, and trees of 64 nodes 67 %.
//
// Softmax.  bf16 and fp32 hold the weights to the same relative precision at any size, so
// the reference of a row need not be its running maximum: it is the maximum of the page
// that set it, and stays until a logit lies 2^kLazy above it.  Only then (and on the first
// page) is there a reduction over the tokens, which lie across lanes; a page otherwise
// costs one vote.  Row sums stay in the lanes until the end of the tile.
// The reference is a score, taken off before the multiplication by scale log2e (a negative
// scale's sign goes into q): the difference of two near scores is exact, and the largest
// weight 1, however large the logits are.  (A fused multiply-add against the rounded product
// as reference is no faster, and off by 2^7 log2 units, a sum of 0 or infinity, at logits of
// 2^31.)
//
// Work.  The pages of all tiles, in order, are cut into equal contiguous ranges, one per
// CTA.  A tile cut by a range's end leaves a partial record (O, reference, sum) in the
// workspace, and a second kernel joins the records of each cut tile.
//
// A CTA goes through its pages in order, all its warps doing the same: their part of V's
// dequantisation, then the softmax (groups of four warps, each some of the rows; one lane a
// token), one barrier a page.  Two more warps issue what is asynchronous: one the products (P V
// of the page before, S of the page ahead, two accumulators), one the copies.  Up to 64 rows a
// tile there are two groups a CTA and two CTAs an SM, which fill each other's waits.  More rows
// share a page's fixed costs (V's dequantisation, the barrier, the products' latency) in tiles of
// 128 by four groups and one CTA an SM: 16 trees of 64 nodes and 16 heads over 4096 to 65536
// tokens take 563 us in tiles of 64, 443 in tiles of 128.  (Warps of fixed roles handing pages to
// each other by barriers, 12 to 20 a CTA, took two to three times as long: each hand-over cost a
// few hundred cycles.)
// All waits are bounded; after one that runs out the CTA goes through its loop without waiting
// or issuing, and the status word says so.
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "score_pipeline.cuh"

namespace mx4 {

namespace tree {

constexpr int kMaxSeq = 256;       // sequences per launch
constexpr float kLazy = 12.f;      // log2 units a logit may lie above its row's reference
constexpr float kUnset = -FLT_MAX;  // the reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKTile = 128 * 128;  // K operand tile
// V operand: rows of 64 dims (128 bytes) a token, in 128-byte swizzle atoms of 8 tokens (the
// 16-byte chunks of row r XOR-permuted by r % 8), 16 atoms, then the other 64 dims.
constexpr int kVTile = 128 * 128 * 2;
constexpr int kVHalf = kVTile / 2;
// P operand: 16-byte chunks of 8 rows, the 128 tokens' chunks one after the other, the next
// 8 rows kChunk bytes on.
constexpr int kChunk = 128 * 16;

// A configuration: NR rows a tile, softmax groups of four warps each, KS and VS stages of K and
// V pages, CTAs an SM.
template <int NR_, int GROUPS_, int KS_, int VS_, int CTAS_>
struct Cfg {
  static constexpr int NR = NR_, KS = KS_, VS = VS_, CTAS = CTAS_;
  static constexpr int NC = NR / GROUPS_;  // rows of a softmax group
  static constexpr int kWorkers = 128 * GROUPS_;   // the threads that compute
  static constexpr int kThreads = kWorkers + 64;   // a warp more for the products, one for the copies
  static constexpr int kVSteps = 16 / (kWorkers / 32);  // V's dequantisation, 8 tokens a warp each
  // hi and lo of q as one operand of 2 NR rows (K read once, their products added by the
  // softmax) while that is cheap there
  static constexpr bool kTwin = NR <= 32;
  static constexpr int kScols = kTwin ? 2 * NR : NR;
  static_assert(NC == 8 || NC == 16 || NC == 32, "rows");
};

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
  int window, sinks;  // (clamped below 2^30: no cached token lies further)
  float cs;     // |scale| log2e (scale 0: 1), finite
  float qsign;  // the scale's sign; 0 for a scale of 0
  uint16_t* out;
  float* lse;
  float* rec;   // [grid][2][NR * 130] partial records
  int32_t* meta;  // [grid][4]
  uint32_t* status;
  int B, N, H, Hkv, G, tiles;
  uint32_t g_inv;  // ceil(2^32 / G)
  // row / G, exact for the rows of a sequence (at most 64 x 128, G at most 128)
  __device__ __forceinline__ int node_of(int row) const {
    return G == 1 ? row : (int)__umulhi((uint32_t)row, g_inv);
  }
};

// Shared-memory layout, in bytes.
template <class C>
struct Lay {
  static constexpr int NR = C::NR;
  static constexpr int kK = 0;                               // [KS] K operand
  static constexpr int kV = kK + C::KS * kKTile;             // V operand
  static constexpr int kP = kV + kVTile;                     // P operand
  static constexpr int kQ = kP + NR / 8 * kChunk;            // q operand: hi, lo
  static constexpr int kKsc = kQ + 2 * NR * 128;             // [KS] K scale words
  static constexpr int kVraw = kKsc + C::KS * 512;           // [VS] V pages as stored
  static constexpr int kSf = kVraw + C::VS * kPageBytes;     // q scale words: hi, lo
  static constexpr int kRef = kSf + 2 * NR * 4;              // [NR] minus the references
  static constexpr int kFac = kRef + NR * 4;                 // [NR] rescaling factors, then 4 / sum
  static constexpr int kWarp = kFac + NR * 4;                // [4][NR] per-warp maxima and sums
  static constexpr int kNan = kWarp + 4 * NR * 4;            // [NR] dim blocks with a visible NaN
  static constexpr int kNode = kNan + NR * 4;                // [NR] output row, -1 none
  static constexpr int kLo = kNode + NR * 4;                 // [NR] first token of the window
  static constexpr int kMask = kLo + NR * 4;                 // [NR] u64: nodes that the row sees
  static constexpr int kPref = kMask + NR * 8;               // [kMaxSeq] u32 page prefix
  static constexpr int kLen = kPref + kMaxSeq * 4;           // [kMaxSeq]
  static constexpr int kCnt = kLen + kMaxSeq * 4;            // [kMaxSeq] u8
  static constexpr int kOff = kCnt + kMaxSeq;                // [4] i64: page offsets of loads
  static constexpr int kBar = kOff + 4 * 8;
  static constexpr int kBars = C::KS + C::VS + 3;
  static constexpr int kStart = kBar + kBars * 8;            // where the range begins
  static constexpr int kInfo = kStart + 24;                  // [4] valid tokens of loaded pages
  static constexpr int kMore = kInfo + 16;                   // [3] a page asks for new references
  static constexpr int kMisc = kMore + 16;                   // abort, tmem address, scan space
  static constexpr int kBytes = kMisc + 8 + 20 * 4 + 1024;    // + slack for the 1024-byte alignment
  static_assert(kV % 1024 == 0 && kVraw % 16 == 0 && kRef % 16 == 0 && kMask % 16 == 0 &&
                kOff % 8 == 0, "alignment");
  static_assert(C::CTAS * (kBytes + 1024) <= 228 * 1024, "shared memory");
};

template <class C>
struct Tm {  // tensor-memory columns
  static constexpr int kS = 0;                    // two S buffers
  static constexpr int kO = 2 * C::kScols;
  static constexpr int kSfa = kO + C::NR;         // two sets (scale fields start at multiples of 4)
  static constexpr int kSfb = kSfa + 8;           // hi, lo
  static constexpr int kSfbRows = C::kTwin ? 2 * C::NR : C::NR;  // rows of one operand
  static constexpr int kSfbW = (kSfbRows + 31) / 32;             // 32 rows a column
  static constexpr int kUsed = kSfb + (C::kTwin ? 4 : 8);
  static_assert(kSfbW <= 4 && kSfa % 4 == 0, "scale fields");
  static constexpr int kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512 && kCols * C::CTAS <= 512, "tensor memory");
};

__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}
// S^T: A e2m1, B e4m3, UE8M0 scales, M = 128, scale byte kb of both words
template <int NR>  // N
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
// Wait for a phase: kSpins tries in a short loop (each sleeps in the hardware for a while).
constexpr int kSpins = 4096, kWaits = 1024;
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
      "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra done;\n"
      " add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra again;\n"
      "done:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "n"(kSpins)
      : "memory");
  return ok != 0u;
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

__device__ __forceinline__ void ld8(uint32_t taddr, float* x) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void st8(uint32_t taddr, const float* x) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(x[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <int W>
__device__ __forceinline__ void ldw(uint32_t taddr, float* x) {
  if constexpr (W == 8) ld8(taddr, x); else ld16(taddr, x);
}
template <int W>
__device__ __forceinline__ void stw(uint32_t taddr, const float* x) {
  if constexpr (W == 8) st8(taddr, x); else st16(taddr, x);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}
// x = (x + y) m
__device__ __forceinline__ void addmul2(float& x0, float& x1, float y0, float y1, uint64_t m) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(pair(x0, x1)), "l"(pair(y0, y1)));
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(r), "l"(m));
  unpair(r, x0, x1);
}
__device__ __forceinline__ void add2(float& x0, float& x1, float y0, float y1) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(pair(x0, x1)), "l"(pair(y0, y1)));
  unpair(r, x0, x1);
}

// The largest of three; a NaN loses.
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
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

// Column sums (maxima) over a warp's lanes of W values a lane: lane l returns column l % W's.
// Each step halves the columns a lane holds: about W shuffles, not 5 W.
template <int W, class Op>
__device__ __forceinline__ float columns(const float* in, int lane, Op op) {
  float v[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = in[i];
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
    }
  }
#pragma unroll
  for (int o = W; o < 32; o <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
  return v[0];
}

// What a sequence's cached tokens give its tiles: pages 0 .. ns-1 hold the first
// `sinks` tokens, pages first .. the window and the drafts.
struct Span {
  int base;  // tokens before the drafts
  int len, n, ns, first, np;
};
__device__ __forceinline__ Span span_of(int L, int n, int window, int sinks) {
  Span sp;
  sp.len = L;
  sp.n = n;
  sp.base = L - n;
  const int lo = window > 0 ? max(0, sp.base + 1 - window) : 0;
  sp.first = lo >> 7;
  sp.ns = min((min(sinks, lo) + kPageTokens - 1) >> 7, sp.first);
  sp.np = n > 0 ? sp.ns + ((L + kPageTokens - 1) >> 7) - sp.first : 0;
  return sp;
}

// floor(U g / G) for g <= G, by one long division
struct Cuts {
  int64_t q;
  uint32_t r, G;
  __device__ __forceinline__ Cuts(int64_t U, uint32_t G_) : G(G_) {
    q = U < (1ll << 32) ? (uint32_t)U / G_ : U / G_;
    r = (uint32_t)(U - q * G_);
  }
  __device__ __forceinline__ int64_t operator()(uint32_t g) const { return q * g + r * g / G; }
};

// Where a CTA's range begins.
struct Start {
  int pages;
  int s, h, rt, e;
};
constexpr int kMinPages = 2;

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::CTAS) tree_kernel(const __grid_constant__ Args a) {
  using L_ = Lay<C>;
  using T_ = Tm<C>;
  constexpr int NR = C::NR, NC = C::NC, KS = C::KS, VS = C::VS, W = NC < 16 ? NC : 16;
  constexpr int kWorkers = C::kWorkers, kThreads = C::kThreads;
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  // (by an offset, not by rounding the pointer: it stays a pointer to shared memory)
  uint8_t* const sm = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
  const uint32_t sb = smem_addr(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* const s_pref = reinterpret_cast<uint32_t*>(sm + L_::kPref);
  int* const s_len = reinterpret_cast<int*>(sm + L_::kLen);
  uint8_t* const s_cnt = sm + L_::kCnt;
  int64_t* const s_off = reinterpret_cast<int64_t*>(sm + L_::kOff);
  int* const s_info = reinterpret_cast<int*>(sm + L_::kInfo);
  Start* const s_start = reinterpret_cast<Start*>(sm + L_::kStart);
  volatile int* const s_abort = reinterpret_cast<volatile int*>(sm + L_::kMisc);
  uint32_t* const s_taddr = reinterpret_cast<uint32_t*>(sm + L_::kMisc + 4);
  uint32_t* const s_scan = reinterpret_cast<uint32_t*>(sm + L_::kMisc + 8);
  auto bar = [&](int i) { return sb + L_::kBar + 8u * i; };
  volatile int* const s_more = reinterpret_cast<volatile int*>(sm + L_::kMore);
  constexpr int kKFull = 0, kVFull = KS, kSFull = KS + VS, kPvDone = kSFull + 2;

  if (tid == 0) {
    for (int i = 0; i < L_::kBars; ++i) mbar_init(bar(i), 1);
    *s_abort = 0;
    s_more[0] = s_more[1] = s_more[2] = 0;
    fence_barrier_init();
  }
  if (tid == kThreads - 32)
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.tmap)) : "memory");
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
  static_assert(kMaxSeq <= kThreads && (int64_t)kMaxSeq << 23 <= 0xFFFFFFFFll, "a thread a sequence");
  {
    uint32_t mine = 0;
    if (tid < a.B) {
      int64_t L = a.seq_lens[tid];
      int n = a.n_nodes ? a.n_nodes[tid] : a.N;
      if (n < 0 || n > a.N || L < n || L > a.bt_width * kPageTokens) {
        if (blockIdx.x == 0) flag(a.status, MX4_STATUS_BAD_LEN);
        n = 0;
        L = 0;
      }
      s_len[tid] = (int)L;
      s_cnt[tid] = (uint8_t)n;
      mine = max(1, span_of((int)L, n, a.window, a.sinks).np);
    }
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += s_scan[w];
    if (tid < a.B) s_pref[tid] = inc;
  }
  __syncthreads();
  // ---- this CTA's range of pages, by one thread (all the divisions are here, once)
  if (tid == 0) {
    const int HT = a.Hkv * a.tiles;
    const int64_t U = (int64_t)s_pref[a.B - 1] * HT;
    // few pages a CTA are not worth the records: at least kMinPages each
    const uint32_t g = blockIdx.x, Gd = (uint32_t)max((int64_t)1, min((int64_t)gridDim.x, U / kMinPages));
    const Cuts cuts(U, Gd);
    Start x{};
    int parts = 0;
    if (g < Gd) {
      const int64_t u0 = cuts(g);
      x.pages = (int)min(cuts(g + 1) - u0, (int64_t)0x7FFFFFFF);
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)s_pref[mid] * HT > u0) hi = mid; else lo = mid + 1;
      }
      const int64_t p0 = lo > 0 ? s_pref[lo - 1] : 0, np = s_pref[lo] - p0, r = u0 - p0 * HT;
      const int ht = r < (1ll << 32) ? (int)((uint32_t)r / (uint32_t)np) : (int)(r / np);
      x.s = lo;
      x.h = ht / a.tiles;
      x.rt = ht % a.tiles;
      x.e = (int)(r - ht * np);
      // a tile that began in the range before this one, and there alone: this CTA's place in
      // the list says how many records join
      const int64_t start = u0 - x.e, end = start + np;
      if (x.e > 0 && cuts(g - 1) <= start) {
        parts = 2;
        while (g + parts - 1 < Gd && cuts(g + parts - 1) < end) ++parts;
        a.meta[4 * g + 1] = x.s;
        a.meta[4 * g + 2] = ht;
      }
    }
    a.meta[4 * g] = parts;
    *s_start = x;
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_launch_dependents();  // after this CTA has its tensor memory

  const uint32_t tm = *s_taddr;
  auto wait = [&](int i, uint32_t parity) -> bool {
    const uint32_t b = bar(i);
    if (__builtin_expect(mbar_spin(b, parity), 1)) return true;
    for (int j = 0; j < kWaits && !*s_abort; ++j)
      if (mbar_spin(b, parity)) return true;
    if (!*s_abort) flag(a.status, MX4_STATUS_TIMEOUT);
    *s_abort = 1;
    return false;
  };

  // (the two branches below pass the same barriers in the same order)
  auto sync_all = []() { asm volatile("bar.sync 1, %0;\n" ::"n"(kThreads) : "memory"); };

  // A place in the list of tiles, and the pages [e0, e1) of the tile in this CTA's range.
  struct Cursor {
    int left;  // pages of the range from e0 on
    int s, h, rt, e0, e1, np;  // np: the tile's places in the list (1 for a tile without pages)
    Span sp;
  };
  auto settle = [&](Cursor& c) {
    if (c.left <= 0) return;
    c.sp = span_of(s_len[c.s], s_cnt[c.s], a.window, a.sinks);
    c.np = max(1, c.sp.np);
    c.e1 = c.e0 + min(c.np - c.e0, c.left);
  };
  auto begin = [&]() {
    Cursor c{s_start->pages, s_start->s, s_start->h, s_start->rt, s_start->e, 0, 0, {}};
    settle(c);
    return c;
  };
  auto advance = [&](Cursor& c) {
    c.left -= c.e1 - c.e0;
    c.e0 = 0;
    if (++c.rt == a.tiles) {
      c.rt = 0;
      if (++c.h == a.Hkv) {
        c.h = 0;
        ++c.s;
      }
    }
    settle(c);
  };
  auto page_no = [](const Span& sp, int e) { return e < sp.ns ? e : sp.first + (e - sp.ns); };

  if (warp == kWorkers / 32 + 1) {
    // ================= the warp of the copies (one lane; all keep step with the barriers)
  // ---- loads, by one thread: page ki of the range is the next K to load, vi the next V.
  // The table entry of page ki is read a page ahead.  A page's offset and its number of valid
  // tokens (0: a bad page, not loaded) are left for V's load and the softmax.
  Cursor lc = begin();
  int ki = 0, vi = 0, le = lc.e0, lpid = -1;
  auto look = [&]() {  // the next page that there is
    while (lc.left > 0 && (le >= lc.e1 || lc.sp.np == 0)) {
      advance(lc);
      le = 0;
    }
    if (lc.left > 0) lpid = a.table[(int64_t)lc.s * a.bt_width + page_no(lc.sp, le)];
  };
  auto load_k = [&]() {
    if (lc.left <= 0 || *s_abort) return;
    const int st = ki % KS;
    const bool ok = lpid >= 0 && lpid < a.num_pages;
    const int64_t off = (int64_t)lpid * a.page_stride + (int64_t)lc.h * a.head_stride;
    s_off[ki & 3] = ok ? off : -1;
    s_info[ki & 3] = ok ? min(kPageTokens, lc.sp.len - page_no(lc.sp, le) * kPageTokens) : 0;
    const uint32_t fb = bar(kKFull + st);
    if (ok) {
      mbar_arrive_expect_tx(fb, kRowDataBytes * kPageTokens + 512);
      asm volatile(
          "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
          "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::"r"(sb + L_::kK + st * kKTile),
          "l"(reinterpret_cast<uint64_t>(&a.tmap)), "r"(0), "r"(0), "r"(0), "r"(lc.h), "r"(lpid),
          "r"(fb)
          : "memory");
      bulk_copy_g2s(sb + L_::kKsc + st * 512, a.k_pages + off + kScaleOffset, 512, fb);
    } else {
      flag(a.status, MX4_STATUS_BAD_PAGE);
      mbar_arrive(fb);
    }
    ++ki;
    ++le;
    look();
  };
  auto load_v = [&]() {
    if (vi >= ki || *s_abort) return;
    const int st = vi % VS;
    const int64_t off = s_off[vi & 3];
    if (off >= 0) {
      mbar_arrive_expect_tx(bar(kVFull + st), kPageBytes);
      bulk_copy_g2s(sb + L_::kVraw + st * kPageBytes, a.v_pages + off, kPageBytes, bar(kVFull + st));
    } else {
      mbar_arrive(bar(kVFull + st));
    }
    ++vi;
  };
  if (lane == 0) {
    look();
    for (int i = 0; i < KS; ++i) load_k();
    for (int i = 0; i < VS; ++i) load_v();
  }

  int k = 0;
  for (Cursor cu = begin(); cu.left > 0; advance(cu)) {
    sync_all();
    sync_all();
    if (cu.sp.np > 0) {
      sync_all();
#pragma unroll 1
      for (int e = cu.e0; e < cu.e1; ++e, ++k) {
        if (lane == 0) {
          if (e > cu.e0) load_v();  // (page k - 1's V has been read)
          wait(kSFull + (k & 1), (k >> 1) & 1);
          load_k();  // (page k's K has been read)
          s_more[(k + 1) % 3] = 0;
          // the workers find the next page's V landed after the barrier, without a wait
          if (VS > 1 && e + 1 < cu.e1) wait(kVFull + (k + 1) % VS, ((k + 1) / VS) & 1);
        }
        __syncwarp();
        if (e == cu.e0) {
          sync_all();
          sync_all();
        }
        sync_all();
        if (s_more[k % 3]) {
          sync_all();
          sync_all();
          sync_all();
        }
      }
      if (lane == 0) load_v();
      __syncwarp();
    }
    sync_all();
    sync_all();
  }
  // after a time-out copies may be under way: none is when the CTA ends
  if (*s_abort && lane == 0) {
    for (int i = max(0, ki - KS); i < ki; ++i)
      for (int j = 0; j < kWaits && !mbar_spin(bar(kKFull + i % KS), (i / KS) & 1); ++j) {}
    for (int i = max(0, vi - VS); i < vi; ++i)
      for (int j = 0; j < kWaits && !mbar_spin(bar(kVFull + i % VS), (i / VS) & 1); ++j) {}
  }
  } else if (warp == kWorkers / 32) {
    // ================= the warp of the products (all lanes go the same way, one issues)
  uint32_t leader;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(leader));
  // S^T = K q^T of page k (K landed: kKFull), fence_after() before
  auto issue_s = [&](int k) {
    const int st = k % KS;
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
                 " @q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(tm + T_::kSfa + 4 * (k & 1)),
                 "l"(desc(sb + L_::kKsc + st * 512, 16, 128)), "r"(leader)
                 : "memory");
    const uint64_t ad = desc(sb + L_::kK + st * kKTile, 16, 1024) | ((uint64_t)2 << 61);
    const uint64_t bd = desc(sb + L_::kQ, 128, 1024);
#pragma unroll
    for (uint32_t part = 0; part < (C::kTwin ? 1 : 2); ++part)
#pragma unroll
      for (uint32_t kb = 0; kb < 4; ++kb)
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 q, %7, 0;\n"
            " @q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, "
            "%2, %3, [%4], [%5], p;\n}\n" ::"r"(tm + T_::kS + (k & 1) * C::kScols),
            "l"(ad + kb * (32 >> 4)), "l"(bd + ((part * NR * 128 + kb * 256) >> 4)),
            "r"(idesc_s<T_::kSfbRows>(kb)), "r"(tm + T_::kSfa + 4 * (k & 1)), "r"(tm + T_::kSfb + part * 4),
            "r"(part + kb), "r"(leader)
            : "memory");
    if (leader) commit(bar(kSFull + (k & 1)));
  };
  // O^T (+)= V^T P^T
  auto issue_pv = [&](bool first) {
    const uint64_t ad = desc(sb + L_::kV, kVHalf, 1024) | ((uint64_t)2 << 61);
    const uint64_t bd = desc(sb + L_::kP, 128, kChunk);
#pragma unroll
    for (uint32_t ks = 0; ks < 8; ++ks)
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
          " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tm + T_::kO),
          "l"(ad + ks * (2048 >> 4)), "l"(bd + ks * (256 >> 4)), "r"(idesc_o<NR>()),
          "r"((uint32_t)(ks > 0 || !first)), "r"(leader)
          : "memory");
    if (leader) commit(bar(kPvDone));
  };


  int k = 0;  // pages done
  for (Cursor cu = begin(); cu.left > 0; advance(cu)) {
    sync_all();  // the tile before is written out
    sync_all();  // rows and q are ready
    if (cu.sp.np > 0) {
      sync_all();  // q's scales are in tensor memory
#pragma unroll 1
      for (int e = cu.e0; e < cu.e1; ++e, ++k) {
        const bool go = !__any_sync(0xFFFFFFFFu, *s_abort);
        if (go) {
          fence_after();
          if (e > cu.e0) issue_pv(e - 1 == cu.e0);
          if (e == cu.e0 && __all_sync(0xFFFFFFFFu, wait(kKFull + k % KS, (k / KS) & 1))) issue_s(k);
          // the next page's S, which the workers find done after the barrier
          if (e + 1 < cu.e1) {
            if (__all_sync(0xFFFFFFFFu, wait(kKFull + (k + 1) % KS, ((k + 1) / KS) & 1)))
              issue_s(k + 1);
            wait(kSFull + ((k + 1) & 1), ((k + 1) >> 1) & 1);
          }
        }
        fence_before();
        if (e == cu.e0) {
          sync_all();
          sync_all();
        }
        sync_all();
        if (s_more[k % 3]) {
          sync_all();
          sync_all();
          sync_all();
        }
      }
      if (!__any_sync(0xFFFFFFFFu, *s_abort)) {
        fence_after();
        issue_pv(cu.e1 - 1 == cu.e0);
      }
    }
    sync_all();  // the sums are there
    sync_all();
  }
  // after a time-out MMAs may be under way: a commit follows all that were issued
  if (*s_abort && leader) {
    const uint32_t b = smem_addr(s_scan);
    mbar_init(b, 1);
    fence_barrier_init();
    commit(b);
    for (int j = 0; j < kWaits && !mbar_spin(b, 0); ++j) {}
  }
  } else {
  // ---- the softmax group's rows c0 .. c0 + NC - 1 of a tile
  const int w = warp & 3, t = tid & 127, c0 = (warp >> 2) * NC;
  const uint32_t tl = tm + ((uint32_t)(32 * w) << 16);
  float* const s_nref = reinterpret_cast<float*>(sm + L_::kRef) + c0;
  float* const s_fac = reinterpret_cast<float*>(sm + L_::kFac) + c0;
  float* const s_warp = reinterpret_cast<float*>(sm + L_::kWarp) + 4 * c0;  // [4][NC]
  uint32_t* const s_nan = reinterpret_cast<uint32_t*>(sm + L_::kNan) + c0;
  int* const s_node = reinterpret_cast<int*>(sm + L_::kNode) + c0;
  int* const s_lo = reinterpret_cast<int*>(sm + L_::kLo) + c0;
  uint32_t* const s_mask = reinterpret_cast<uint32_t*>(sm + L_::kMask) + 2 * c0;  // [2][NC]
  const uint64_t cs2 = pair(a.cs, a.cs);
  const int tok = 4 * lane + w;  // this lane's token of a page
  // dequantisation: see below
  const int r8 = lane & 7, blk = ((r8 >> 1) + (lane >> 3)) & 3;

  // A tile's q: 16 elements a thread, K-chunk j of row n (the two threads of a 32-block share
  // its largest magnitude), on their way while the tile before is written out.
  constexpr int kQIt = (NR * 8 + kWorkers - 1) / kWorkers;
  uint4 qx[kQIt][2];
  auto fetch_q = [&](const Cursor& c) {
#pragma unroll
    for (int it = 0; it < kQIt; ++it) {
      const int n = (tid >> 3) + it * (kWorkers / 8), row = c.rt * NR + n, node = a.node_of(row);
      qx[it][0] = qx[it][1] = make_uint4(0u, 0u, 0u, 0u);
      if (n < NR && c.left > 0 && node < c.sp.n) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (((int64_t)c.s * a.N + node) * a.H + c.h * a.G + (row - node * a.G)) * kHeadDim +
            16 * (tid & 7));
        qx[it][0] = src[0];
        qx[it][1] = src[1];
      }
    }
  };

  int k = 0;  // pages done
  Cursor cu = begin();
  fetch_q(cu);
  while (cu.left > 0) {
    const Span sp = cu.sp;
    const bool begins = cu.e0 == 0, ends = cu.e1 >= sp.np;
    sync_all();  // the tile before is written out
    // ---- the tile's rows
    if (t < NC) {
      const int row = cu.rt * NR + c0 + t, node = a.node_of(row);
      s_node[t] = node < a.N ? node * a.H + cu.h * a.G + (row - node * a.G) : -1;
      uint64_t mk = 0;
      int lo = 0;
      if (node < sp.n) {
        const uint64_t all = sp.n < 64 ? (1ull << sp.n) - 1 : ~0ull;
        auto mask_of = [&](int j) {
          return (a.mask ? a.mask[(int64_t)cu.s * a.N + j] : (2ull << j) - 1) & all;
        };
        mk = mask_of(node);
        if (a.window > 0) {
          const int d = max(1, __popcll(mk)) - 1;
          lo = max(0, sp.base + d + 1 - a.window);
          // (nodes' depths differ by less than n: none leaves a window that is not shorter)
#pragma unroll 1
          for (int i = 0; i < (a.window < sp.n ? sp.n : 0); ++i) {
            const int di = max(1, __popcll(mask_of(i))) - 1;
            if (!(di > d - a.window || sp.base + di < a.sinks)) mk &= ~(1ull << i);
          }
        }
      }
      s_mask[t] = (uint32_t)mk;
      s_mask[NC + t] = (uint32_t)(mk >> 32);
      s_lo[t] = lo;
      s_nref[t] = -kUnset;
      s_nan[t] = 0;
    }
    // ---- q
    if (sp.np > 0) {
#pragma unroll
      for (int it = 0; it < kQIt; ++it) {
        const int n = (tid >> 3) + it * (kWorkers / 8), j = tid & 7;
        if (n >= NR) break;
        const uint4 x0 = qx[it][0], x1 = qx[it][1];
        const uint32_t wd[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        float amax = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_float(wd[u] & 0xFFFFu)),
                                   fabsf(bf16_bits_to_float(wd[u] >> 16))));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        const int ef = min(254, (int)(__float_as_uint(amax) >> 23));
        const int E = amax == 0.f ? 0 : max(-122, ef - 127 - 7);
        const float inv = __uint_as_float((uint32_t)(127 - E) << 23) * a.qsign;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint16_t hc[2], lc2[2];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t x2 = wd[2 * u + v];
            float y0 = bf16_bits_to_float(x2 & 0xFFFFu), y1 = bf16_bits_to_float(x2 >> 16);
            // an infinity has no E4M3 code: NaN, as its logits would be
            y0 = isinf(y0) ? NAN : y0 * inv;
            y1 = isinf(y1) ? NAN : y1 * inv;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n" : "=h"(hc[v]) : "f"(y0), "f"(y1));
            uint32_t hf;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(hf) : "h"(hc[v]));
            const float h0 = __half2float(__ushort_as_half((unsigned short)(hf & 0xFFFFu)));
            const float h1 = __half2float(__ushort_as_half((unsigned short)(hf >> 16)));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n"
                : "=h"(lc2[v])
                : "f"((y0 - h0) * 32.f), "f"((y1 - h1) * 32.f));
          }
          hi[u] = (uint32_t)hc[0] | ((uint32_t)hc[1] << 16);
          lo[u] = (uint32_t)lc2[0] | ((uint32_t)lc2[1] << 16);
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
    }
    sync_all();
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;

    if (sp.np > 0) {
      // operand row n's scale word at lane n % 32 of every lane quarter, column n / 32
      if (warp < 4) {
#pragma unroll
        for (int part = 0; part < (C::kTwin ? 1 : 2); ++part)
#pragma unroll
          for (int c = 0; c < T_::kSfbW; ++c)
            st1(tl + T_::kSfb + part * 4 + c,
                *reinterpret_cast<const uint32_t*>(sm + L_::kSf + (part * NR + c * 32 + lane) * 4));
        wait_st();
      }
      fence_before();
      sync_all();
#pragma unroll 1
      for (int e = cu.e0; e < cu.e1; ++e, ++k) {
        const int first = page_no(sp, e) * kPageTokens, live = s_info[k & 3];
        const bool plain = live == kPageTokens && first + kPageTokens <= sp.base &&
                           (a.window == 0 || first >= sp.base + sp.n - a.window ||
                            first + kPageTokens <= a.sinks);
        // ---- V.  Operand row (K index) m holds token 4 (m % 32) + m / 32, the order in which
        // the tensor copy lays out K.  A warp's step: 8 operand rows (r8), lane >> 3 choosing
        // which 32-dim block of each: 16 raw bytes a lane, four 16-byte stores without bank
        // conflicts.
        auto convert_v = [&](int it, uint32_t (&y)[4][4]) {
          const uint8_t* raw = sm + L_::kVraw + (k % VS) * kPageBytes;
          const int m = (warp * C::kVSteps + it) * 8 + r8, tk = 4 * (m & 31) + (m >> 5);
          const uint4 c4 = *reinterpret_cast<const uint4*>(raw + tk * kRowDataBytes + blk * 16);
          const uint32_t sc = raw[kScaleOffset + tk * kRowScaleBytes + blk];
          const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
          // 2^(sc - 3), as two factors where it passes bf16's range
          const uint32_t f1 = (tk < live && sc != 255u ? min(sc + 124u, 254u) : 0u) * 0x00800080u;
          const bool big = __any_sync(0xFFFFFFFFu, sc > 130u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v = cw[j];
            // Codes i and i + 4 of the word as one pair: a code's four bits to places 15 .. 12
            // and 9 .. 6 by one multiplication (on the FMA pipe, which has twice the logic
            // pipe's rate), then its sign from the one and the other three from the other.
            const uint32_t u = v >> 8;
            y[j][0] = ((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
            y[j][1] = ((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
            y[j][2] = ((u & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
            y[j][3] = ((u & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[j][i] = bf16_mul2(y[j][i], f1);
          }
          if (big) {
            const uint32_t f2 = (sc > 130u ? sc - 3u : 127u) * 0x00800080u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) y[j][i] = bf16_mul2(y[j][i], f2);
          }
        };
        auto store_v = [&](int it, const uint32_t (&y)[4][4]) {
          const int m = (warp * C::kVSteps + it) * 8 + r8;
          uint8_t* const dst = sm + L_::kV + (blk >> 1) * kVHalf + (m >> 3) * 1024 + r8 * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(dst + ((((blk & 1) * 4 + j) ^ r8) << 4)) =
                make_uint4(y[j][0], y[j][1], y[j][2], y[j][3]);
        };
        // The operands' buffers are free once the product of the page before is done.  With two
        // stages of V its first half is converted before that, else (V lands last) the weights
        // are computed before.
        uint32_t yv[4][4];
        if (VS > 1 && e == cu.e0) wait(kVFull + k % VS, (k / VS) & 1);
        if constexpr (VS > 1) {
          convert_v(0, yv);
          if (k > 0) wait(kPvDone, (k - 1) & 1);
          store_v(0, yv);
          if constexpr (C::kVSteps > 1) {
            convert_v(1, yv);
            store_v(1, yv);
          }
        }
        // ---- scores, their differences from the rows' references in log2 units
        // a row sees a draft by its mask, an earlier token from the window's first on; rows
        // without a node see what they like, their results are zeroed
        uint32_t vis = ~0u;
        if (!plain) {
          vis = 0u;
          const int i_g = first + tok, nd = i_g - sp.base;
          if (tok < live && nd >= 0) {
            const uint32_t* const mw = s_mask + ((nd >> 5) & 1) * NC;
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
              const uint4 m4 = *reinterpret_cast<const uint4*>(mw + c);
              const uint32_t mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) vis |= ((mm[i] >> (nd & 31)) & 1u) << (c + i);
            }
          } else if (tok < live) {
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
              const int4 l4 = *reinterpret_cast<const int4*>(s_lo + c);
              const int lo[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) vis |= (uint32_t)(i_g >= lo[i]) << (c + i);
            }
            if (i_g < a.sinks) vis = ~0u;
          }
        }
        if (e == cu.e0) wait(kSFull + (k & 1), (k >> 1) & 1);
        fence_after();
        const uint32_t ts = tl + T_::kS + (k & 1) * C::kScols + c0;
        // S of W rows, hi and lo parts added where they are apart
        auto s_of = [&](int c, float* v) {
          ldw<W>(ts + c, v);
          if constexpr (C::kTwin) {
            float z[W];
            ldw<W>(ts + NR + c, z);
            wait_ld();
#pragma unroll
            for (int i = 0; i < W; i += 2) add2(v[i], v[i + 1], z[i], z[i + 1]);
          } else {
            wait_ld();
          }
        };
        // -inf where not seen, whatever was computed there
        auto hide = [&](int c, float* v) {
          if (plain) return;
          const uint32_t vb = vis >> c;
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] = (vb >> i) & 1u ? v[i] : -INFINITY;
        };
        // The weights of the page, into the P operand and the row sums, W rows at a time.  Where
        // a logit lies too far above its reference, those W rows' weights are not summed yet
        // (owed): the page is taken again with new references.  What was summed is right in
        // either case, it is brought to the new references with the rest.  A tile's first page
        // starts with them.
        uint32_t owed = ~0u;
        uint8_t* const pd = sm + L_::kP + (c0 >> 3) * kChunk + (4 * w + (lane >> 3)) * 128 + (lane & 7) * 16;
        uint32_t pk[NC / 2];
        bool renew = e == cu.e0;
#pragma unroll 1
        for (int round = 0;; ++round) {
          if (renew) {
            // The page's maximum of each row that has a larger one; what was summed so far is
            // brought to them.  (The product of the page before is done, its buffers were free
            // above; this page's waits for the round's last barrier.)
            fence_after();
#pragma unroll 1
            for (int c = 0; c < NC; c += W) {
              float v[W];
              s_of(c, v);
              hide(c, v);
              const float mx = columns<W>(v, lane, [](float p, float q) { return fmaxf(p, q); });
              if (lane < W) s_warp[w * NC + c + lane] = mx;
            }
            sync_all();
            if (t < NC) {
              const float v = fmaxf(fmaxf(s_warp[t], s_warp[NC + t]),
                                    fmaxf(s_warp[2 * NC + t], s_warp[3 * NC + t]));
              const float old = -s_nref[t], now = fmaxf(old, v);
              s_fac[t] = ex2((old - now) * a.cs);
              s_nref[t] = -now;
            }
            sync_all();
            if (e > cu.e0 || round > 0) {
#pragma unroll
              for (int c = 0; c < NC; ++c) l[c] *= s_fac[c];
            }
            if (e > cu.e0) {
#pragma unroll 1
              for (int c = 0; c < NC; c += W) {
                float o[W];
                ldw<W>(tl + T_::kO + c0 + c, o);
                wait_ld();
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] *= s_fac[c + i];
                stw<W>(tl + T_::kO + c0 + c, o);
              }
              wait_st();
            }
          }
#pragma unroll
          for (int c = 0; c < NC; c += W) {
            float x[W];
            s_of(c, x);
#pragma unroll
            for (int i = 0; i < W; i += 4) {
              const float4 rf = *reinterpret_cast<const float4*>(s_nref + c + i);
              addmul2(x[i], x[i + 1], rf.x, rf.y, cs2);
              addmul2(x[i + 2], x[i + 3], rf.z, rf.w, cs2);
            }
            hide(c, x);
            float m0 = x[0], m1 = x[1];
#pragma unroll
            for (int i = 2; i + 3 < W; i += 4) {
              m0 = max3(m0, x[i], x[i + 1]);
              m1 = max3(m1, x[i + 2], x[i + 3]);
            }
            m0 = max3(m0, m1, fmaxf(x[W - 2], x[W - 1]));
            const bool far = __any_sync(0xFFFFFFFFu, m0 > kLazy);
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = ex2(x[i]);
            if ((owed >> c) & 1u) {
              if (far && round == 0) {
                if (lane == 0) s_more[k % 3] = 1;
              } else {
#pragma unroll
                for (int i = 0; i < W; i += 2) add2(l[c + i], l[c + i + 1], x[i], x[i + 1]);
                owed &= ~(1u << c);
              }
            }
#pragma unroll
            for (int i = 0; i < W; i += 2) pk[(c + i) / 2] = pack_bf16(x[i], x[i + 1]);
          }
          if (VS == 1 && round == 0 && k > 0) wait(kPvDone, (k - 1) & 1);
#pragma unroll
          for (int c = 0; c < NC; c += 8)
            *reinterpret_cast<uint4*>(pd + (c >> 3) * kChunk) =
                make_uint4(pk[c / 2], pk[c / 2 + 1], pk[c / 2 + 2], pk[c / 2 + 3]);
          if (round == 0) {
            if constexpr (VS == 1) {
              wait(kVFull + k % VS, (k / VS) & 1);
#pragma unroll
              for (int it = 0; it < C::kVSteps; ++it) {
                convert_v(it, yv);
                store_v(it, yv);
              }
            }
            // NaN dim blocks of this lane's token
            uint32_t vw = *reinterpret_cast<const uint32_t*>(
                sm + L_::kVraw + (k % VS) * kPageBytes + kScaleOffset + tok * kRowScaleBytes);
            vw = ((vw & 0x7F7F7F7Fu) + 0x01010101u) & vw & 0x80808080u;
            if (vw != 0u && tok < live) {  // the rows that see the token get its NaNs at the end
    #pragma unroll 1
              for (int c = 0; c < NC; ++c)
                if ((vis >> c) & 1u) atomicOr(s_nan + c, vw);
            }
          }
          fence_async();
          fence_before();
          sync_all();
          if (round > 0 || !s_more[k % 3]) break;
          renew = true;
        }
      }
      Cursor nx = cu;
      advance(nx);
      fetch_q(nx);
#pragma unroll
      for (int c = 0; c < NC; c += W) {
        const float v = columns<W>(l + c, lane, [](float p, float q) { return p + q; });
        if (lane < W) s_warp[w * NC + c + lane] = v;
      }
      wait(kPvDone, (k - 1) & 1);
    } else {
#pragma unroll 1
      for (int c = t; c < 4 * NC; c += 128) s_warp[c] = 0.f;
    }
    sync_all();
    // ---- the tile's result: this lane's dim of every row
    const bool whole = begins && ends;
    float* const rec = a.rec + (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * (int64_t)(NR * 130);
    if (t < NC) {
      float sum = (s_warp[t] + s_warp[NC + t]) + (s_warp[2 * NC + t] + s_warp[3 * NC + t]);
      if (a.node_of(cu.rt * NR + c0 + t) >= sp.n) sum = 0.f;
      const float rf = -s_nref[t];
      if (whole) {
        s_fac[t] = sum == 0.f ? 0.f : 4.f / sum;
        if (a.lse && s_node[t] >= 0)
          a.lse[(int64_t)cu.s * a.N * a.H + s_node[t]] =
              sum == 0.f ? -INFINITY : (log2f(sum) + rf * a.cs) * 0.6931471805599453f;
      } else {
        s_fac[t] = sum == 0.f ? 0.f : 1.f;
        rec[NR * 128 + c0 + t] = rf;
        rec[NR * 129 + c0 + t] = sum;
      }
    }
    sync_all();
    fence_after();
    // operand position -> dim: the codes of a word were paired i, i + 4
    const int dim = 32 * w + (lane & 24) + ((lane & 1) << 2) + ((lane & 7) >> 1);
    const uint32_t nb = 0x80u << (8 * w);
    uint16_t* const out = a.out + (int64_t)cu.s * a.N * a.H * kHeadDim + dim;
    float* const orec = rec + c0 * 128 + dim;
#pragma unroll 1
    for (int c = 0; c < NC; c += W) {
      float o[W];
      if (sp.np > 0) {
        ldw<W>(tl + T_::kO + c0 + c, o);
        wait_ld();
      }
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const float4 f4 = *reinterpret_cast<const float4*>(s_fac + c + i);
        const uint4 n4 = *reinterpret_cast<const uint4*>(s_nan + c + i);
        const float f[4] = {f4.x, f4.y, f4.z, f4.w};
        const uint32_t nn[4] = {n4.x, n4.y, n4.z, n4.w};
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] = sp.np == 0 || f[u] == 0.f ? 0.f : (nn[u] & nb) ? NAN : o[i + u] * f[u];
        if (whole) {
          const int4 r4 = *reinterpret_cast<const int4*>(s_node + c + i);
          const int row[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (row[u] >= 0)
              out[row[u] * kHeadDim] = __bfloat16_as_ushort(__float2bfloat16_rn(v[u]));
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) orec[(c + i + u) * 128] = v[u];
        }
      }
    }
    fence_before();
    if (sp.np == 0) {
      Cursor nx = cu;
      advance(nx);
      fetch_q(nx);
    }
    advance(cu);
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
// a lane four dims: out = 4 sum_r O_r f_r / sum_r l_r f_r with f_r = 2^(cs (m_r - M)).
template <int NR>
__global__ void __launch_bounds__(128) tree_merge_kernel(const Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t g = blockIdx.x;
  const int parts = a.meta[4 * g];
  if (parts < 2) return;
  const int s = a.meta[4 * g + 1], ht = a.meta[4 * g + 2];
  const int h = ht / a.tiles, rt = ht % a.tiles, lane = threadIdx.x & 31;
  const int c = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int row = rt * NR + c, node = a.node_of(row);
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
    const float f = ex2((m - M) * a.cs);
    sum = fmaf(l, f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  const int64_t o = ((int64_t)s * a.N + node) * a.H + h * a.G + (row - node * a.G);
  const float f = sum == 0.f ? 0.f : 4.f / sum;
  uint2 y;
  y.x = pack_bf16(f == 0.f ? 0.f : acc.x * f, f == 0.f ? 0.f : acc.y * f);
  y.y = pack_bf16(f == 0.f ? 0.f : acc.z * f, f == 0.f ? 0.f : acc.w * f);
  reinterpret_cast<uint2*>(a.out + o * kHeadDim)[lane] = y;
  if (a.lse && lane == 0)
    a.lse[o] = sum == 0.f ? -INFINITY : (log2f(sum) + M * a.cs) * 0.6931471805599453f;
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

template <class C>
cudaError_t launch(Args a, int64_t B, int num_sms, cudaStream_t stream) {
  const int smem = Lay<C>::kBytes;
  auto kern = tree_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = num_sms * C::CTAS;
  a.tiles = (a.N * a.G + C::NR - 1) / C::NR;
  a.meta = reinterpret_cast<int32_t*>(a.rec + (int64_t)grid * 2 * C::NR * 130);
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
    e = launch_pdl(kern, dim3(grid), dim3(C::kThreads), smem, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tree_merge_kernel<C::NR>, dim3(grid, C::NR / 4), dim3(128), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Rows a tile: the smallest that holds all of a sequence's rows of one KV head, else the
// largest.  (Three stages of K at 128 rows: 443 us for 456 with two.)
//               NR groups KS VS CTAs
using C16 = Cfg<16, 2, 2, 2, 2>;
using C32 = Cfg<32, 2, 2, 2, 2>;
using C64 = Cfg<64, 2, 2, 1, 2>;
using C128 = Cfg<128, 4, 3, 2, 1>;
inline int rows_of(int N, int H, int Hkv) {
  const int rows = N * (H / Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}
inline int ctas_of(int nr) {
  return nr == 16 ? C16::CTAS : nr == 32 ? C32::CTAS : nr == 64 ? C64::CTAS : C128::CTAS;
}

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
  a.window = (int)std::min<int64_t>(window, 1 << 30);
  a.sinks = (int)std::min<int64_t>(sinks, 1 << 30);
  a.cs = scale == 0.f ? 1.f : std::min(std::fabs(scale) * tree::kLog2e, FLT_MAX);
  a.qsign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
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
  a.g_inv = (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
  a.tiles = 0;
  if (cudaError_t e = tree::encode_pool(k_pages, page_stride, head_stride, num_pages, Hkv, &a.tmap))
    return e;
  switch (tree::rows_of(N, H, Hkv)) {
    case 16: return tree::launch<tree::C16>(a, B, num_sms, stream);
    case 32: return tree::launch<tree::C32>(a, B, num_sms, stream);
    case 64: return tree::launch<tree::C64>(a, B, num_sms, stream);
    default: return tree::launch<tree::C128>(a, B, num_sms, stream);
  }
}

}  // namespace mx4
