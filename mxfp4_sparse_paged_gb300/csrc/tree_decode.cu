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
// Roles.  Warps 0 and 3 stream the pages' K (tensor copies into the operand's swizzled
// layout) and V (bulk copies), warps 1 and 2 issue the two products, then come the softmax
// warps (groups of four, one lane a token, each group its own rows; in the epilogue one lane
// a dim) and the warps that convert q and dequantise V.  All waits are bounded; after one
// that runs out every role goes through its loop without waiting or issuing, and the status
// word says so.
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled
#include <cuda_bf16.h>

#include <algorithm>

#include "score_pipeline.cuh"

namespace mx4 {

namespace tree {

constexpr int kMaxSeq = 256;       // sequences per launch
constexpr float kLazy = 12.f;      // log2 units a logit may lie above its row's reference
constexpr float kUnset = -3e38f;   // the reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKTile = 128 * 128;  // K operand tile
// V operand: rows of 64 dims (128 bytes) a token, in 128-byte swizzle atoms of 8 tokens (the
// 16-byte chunks of row r XOR-permuted by r % 8), 16 atoms, then the other 64 dims.
constexpr int kVTile = 128 * 128 * 2;
constexpr int kVHalf = kVTile / 2;
// P operand: 16-byte chunks of 8 rows, the 128 tokens' chunks one after the other, the next
// 8 rows kChunk bytes on (16 more than the chunks take, to change banks).
constexpr int kChunk = 128 * 16 + 16;

// A configuration: NR rows a tile, SG softmax groups (of NR / SG rows), DW dequantising
// warps, KS and VS stages of K and V pages, VB operand buffers of V and P, CTAs an SM.
// Registers are dealt out by role (RC: control warps, RS: softmax, RD: dequantisation), in
// place of the same number for all.
template <int NR_, int SG_, int DW_, int KS_, int VS_, int VB_, int CTAS_, int RC_, int RS_, int RD_>
struct Cfg {
  static constexpr int NR = NR_, SG = SG_, DW = DW_, KS = KS_, VS = VS_, VB = VB_, CTAS = CTAS_;
  static constexpr int RC = RC_, RS = RS_, RD = RD_;
  static_assert(VB <= 2 && NR <= 32 * SG && DW % 4 == 0 && NR % (16 * SG) == 0, "whole warpgroups, 16 rows at a time");
  static constexpr int kRegs = 128 * (RC + SG * RS + DW / 4 * RD);  // all that the roles take
  static constexpr int NC = NR / SG;
  static constexpr int kThreads = 32 * (4 + 4 * SG + DW);
  // hi and lo of q as one operand of 2 NR rows (K read once, their products added by the
  // softmax) while that is cheap there
  static constexpr bool kTwin = NR <= 32;
  static constexpr int kScols = kTwin ? 2 * NR : NR;
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
  float scale;
  uint16_t* out;
  float* lse;
  float* rec;   // [grid][2][NR * 130] partial records
  int32_t* meta;  // [grid][4]
  uint32_t* status;
  int B, N, H, Hkv, G, tiles;
};

// Shared-memory layout, in bytes.
template <class C>
struct Lay {
  static constexpr int NR = C::NR;
  static constexpr int kK = 0;                               // [KS] K operand
  static constexpr int kV = kK + C::KS * kKTile;             // [VB] V operand
  static constexpr int kKsc = kV + C::VB * kVTile;           // [KS] scale words: K's, V's
  static constexpr int kVraw = kKsc + C::KS * 1024;           // [VS] V pages as stored
  static constexpr int kP = kVraw + C::VS * kPageBytes;      // [VB] P operand
  static constexpr int kQ = (kP + C::VB * (NR / 8) * kChunk + 127) / 128 * 128;           // q operand: hi, lo
  static constexpr int kSf = kQ + 2 * NR * 128;              // q scale words: hi, lo
  static constexpr int kRef = kSf + 2 * NR * 4;              // [NR] minus the references
  static constexpr int kFac = kRef + NR * 4;                 // [NR] rescaling factors, then 1 / sum
  static constexpr int kWarp = kFac + NR * 4;                // [4][NR] per-warp maxima and sums
  static constexpr int kNan = kWarp + 4 * NR * 4;            // [NR] dim blocks with a visible NaN
  static constexpr int kNode = kNan + NR * 4;                // [NR] output row, -1 none
  static constexpr int kLo = kNode + NR * 4;                 // [NR] first token of the window
  static constexpr int kMask = kLo + NR * 4;                 // [NR] u64: nodes that the row sees
  static constexpr int kPref = kMask + NR * 8;               // [kMaxSeq] i64 page prefix
  static constexpr int kLen = kPref + kMaxSeq * 8;           // [kMaxSeq]
  static constexpr int kCnt = kLen + kMaxSeq * 4;            // [kMaxSeq] u8
  static constexpr int kInfo = kCnt + kMaxSeq;               // [VS] valid tokens of the page
  static constexpr int kKinfo = kInfo + C::VS * 4;           // [KS] the same
  static constexpr int kBar = (kKinfo + C::KS * 4 + 7) / 8 * 8;
  static constexpr int kBars = 2 * C::KS + 2 * C::VS + 4 + 3 * C::VB + 5;
  static constexpr int kStart = kBar + kBars * 8;            // where the range begins
  static constexpr int kMisc = kStart + 24;                  // abort, tmem address, scan space
  static constexpr int kBytes = kMisc + 16 + 32 * 8 + 1024;  // + slack for the 1024-byte alignment
  static_assert(kVraw % 16 == 0 && kV % 1024 == 0 && kP % 16 == 0 && kQ % 128 == 0 && kRef % 16 == 0 && kMask % 8 == 0, "alignment");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <class C>
struct Tm {  // tensor-memory columns
  static constexpr int kS = 0;                    // two S buffers
  static constexpr int kO = 2 * C::kScols;
  static constexpr int kSfa = kO + C::NR;         // two sets of 4 (scale fields start at
  static constexpr int kSfb = kSfa + 8;           // multiples of 4)
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
// A ring position: slot and the parity of its use.
template <int S>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// This warpgroup's registers a thread from here on.
template <int kFrom, int kTo>
__device__ __forceinline__ void set_regs() {
  if constexpr (kTo > kFrom)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kTo));
  else if constexpr (kTo < kFrom)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kTo));
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

__host__ __device__ __forceinline__ int64_t range_begin(int64_t g, int64_t U, int64_t G) {
  return U * g / G;
}

// Where a CTA's range begins.
struct Start {
  int64_t pages;
  int s, h, rt, e;
};
constexpr int kMinPages = 2;

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::CTAS) tree_kernel(const __grid_constant__ Args a) {
  using L_ = Lay<C>;
  using T_ = Tm<C>;
  constexpr int NR = C::NR, NC = C::NC, SG = C::SG, DW = C::DW, KS = C::KS, VS = C::VS, VB = C::VB;
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t* const s_pref = reinterpret_cast<int64_t*>(sm + L_::kPref);
  int* const s_len = reinterpret_cast<int*>(sm + L_::kLen);
  uint8_t* const s_cnt = sm + L_::kCnt;
  volatile int* const s_info = reinterpret_cast<volatile int*>(sm + L_::kInfo);
  volatile int* const s_kinfo = reinterpret_cast<volatile int*>(sm + L_::kKinfo);
  volatile int* const s_abort = reinterpret_cast<volatile int*>(sm + L_::kMisc);
  uint32_t* const s_taddr = reinterpret_cast<uint32_t*>(sm + L_::kMisc + 4);
  int64_t* const s_scan = reinterpret_cast<int64_t*>(sm + L_::kMisc + 16);
  auto bar = [&](int i) { return sb + L_::kBar + 8u * i; };
  constexpr int kKFull = 0, kKEmpty = KS, kVFull = 2 * KS, kVEmpty = kVFull + VS,
                kSFull = kVEmpty + VS, kSFree = kSFull + 2, kPFull = kSFree + 2,
                kVReady = kPFull + VB, kPvDone = kVReady + VB, kQFull = kPvDone + VB,
                kQEmpty = kQFull + 1, kOFree = kQEmpty + 1, kDrain = kOFree + 1;  // two

  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(bar(kKFull + i), 1);
      mbar_init(bar(kKEmpty + i), 1 + 4 * SG);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(bar(kVFull + i), 1);
      mbar_init(bar(kVEmpty + i), DW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kSFree + i), 4 * SG);
      mbar_init(bar(kDrain + i), 1);
    }
    for (int i = 0; i < VB; ++i) {
      mbar_init(bar(kPFull + i), 4 * SG);
      mbar_init(bar(kVReady + i), DW);
      mbar_init(bar(kPvDone + i), 1);
    }
    mbar_init(bar(kQFull), DW);
    mbar_init(bar(kQEmpty), 1);
    mbar_init(bar(kOFree), 4 * SG);
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
    static_assert(kMaxSeq <= C::kThreads, "a thread a sequence");
    int64_t mine = 0;
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
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += s_scan[w];
    if (tid < a.B) s_pref[tid] = inc;
  }
  __syncthreads();
  // ---- this CTA's range of pages, by one thread (all the divisions are here, once)
  Start* const s_start = reinterpret_cast<Start*>(sm + L_::kStart);
  if (tid == 0) {
    const int HT = a.Hkv * a.tiles;
    const int64_t U = s_pref[a.B - 1] * HT, g = blockIdx.x;
    // few pages a CTA are not worth the records: at least kMinPages each
    const int64_t Gd = max((int64_t)1, min((int64_t)gridDim.x, U / kMinPages));
    Start x{};
    int parts = 0;
    if (g < Gd) {
      const int64_t u0 = range_begin(g, U, Gd);
      x.pages = range_begin(g + 1, U, Gd) - u0;
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] * HT > u0) hi = mid; else lo = mid + 1;
      }
      const int64_t p0 = lo > 0 ? s_pref[lo - 1] : 0, np = s_pref[lo] - p0, r = u0 - p0 * HT;
      const int ht = (int)(r / np);
      x.s = lo;
      x.h = ht / a.tiles;
      x.rt = ht % a.tiles;
      x.e = (int)(r - ht * np);
      // a tile that began in the range before this one, and there alone: this CTA's place in
      // the list says how many records join
      const int64_t start = u0 - x.e, end = start + np;
      if (x.e > 0 && range_begin(g - 1, U, Gd) <= start) {
        parts = 2;
        while (g + parts - 1 < Gd && range_begin(g + parts - 1, U, Gd) < end) ++parts;
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

  // A place in the list of tiles, and the pages [e0, e1) of the tile in this CTA's range.
  struct Cursor {
    int64_t left;  // pages of the range from e0 on
    int s, h, rt, e0, e1, np;  // np: the tile's places in the list (1 for a tile without pages)
    Span sp;
  };
  auto settle = [&](Cursor& c) {
    if (c.left <= 0) return;
    c.sp = span_of(s_len[c.s], s_cnt[c.s], a.window, a.sinks);
    c.np = max(1, c.sp.np);
    c.e1 = (int)min((int64_t)c.np, c.e0 + c.left);
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
  // The tiles of this CTA's range, in order: f(tile number among those with pages, sequence,
  // head, row tile, its span, its pages [e0, e1) of this range).
  auto for_tiles = [&](auto&& f) {
    int count = 0;
    for (Cursor c = begin(); c.left > 0; advance(c)) {
      f(count, c.s, c.h, c.rt, c.sp, c.e0, c.e1);
      count += c.sp.np > 0;
    }
  };
  auto page_no = [](const Span& sp, int e) { return e < sp.ns ? e : sp.first + (e - sp.ns); };

  constexpr int kLaunchRegs = 65536 / (C::CTAS * C::kThreads) / 8 * 8;
  static_assert(C::kRegs <= kLaunchRegs * C::kThreads, "the roles' registers are the launch's");
  if (warp < 4) {
  set_regs<kLaunchRegs, C::RC>();  // (by the warpgroup as one)
  if (warp == 0 || warp == 3) {
    // ================= producers: K (warp 0) and V (warp 3).  The lanes look up 32 pages of a
    // tile at once, the next ones before the present ones' copies.
    const bool isv = warp == 3;
    int k = 0;
    Ring<KS> kr;
    Ring<VS> vr;
    Cursor c = begin();
    auto look = [&](const Cursor& x) {
      const int e = x.e0 + lane;
      return x.left > 0 && x.sp.np > 0 && e < x.e1
                 ? a.table[(int64_t)x.s * a.bt_width + page_no(x.sp, e)]
                 : -1;
    };
    int pid_n = look(c);
    while (c.left > 0) {
      const Cursor cur = c;
      const int pid_c = pid_n;
      const int cnt = min(32, cur.e1 - cur.e0);
      if (cnt < cur.e1 - cur.e0) {
        c.e0 += 32;
        c.left -= 32;
      } else {
        advance(c);
      }
      pid_n = look(c);
      if (cur.sp.np == 0) continue;
#pragma unroll 1
      for (int i = 0; i < cnt; ++i) {
        const int pid = __shfl_sync(0xFFFFFFFFu, pid_c, i);
        if (lane == 0) {
          const bool ok = pid >= 0 && pid < a.num_pages;
          const int live = min(kPageTokens, cur.sp.len - page_no(cur.sp, cur.e0 + i) * kPageTokens);
          const int64_t off = (int64_t)pid * a.page_stride + (int64_t)cur.h * a.head_stride;
          const int st = isv ? vr.slot : kr.slot;
          const uint32_t fb = bar((isv ? kVFull : kKFull) + st);
          bool go = !*s_abort;
          if (k >= (isv ? VS : KS))
            go = wait((isv ? kVEmpty : kKEmpty) + st, (isv ? vr.phase : kr.phase) ^ 1u) && go;
          if (go) {
            if (isv) s_info[st] = ok ? live : 0; else s_kinfo[st] = ok ? live : 0;
            if (!ok) {
              flag(a.status, MX4_STATUS_BAD_PAGE);
              mbar_arrive(fb);
            } else if (isv) {
              mbar_arrive_expect_tx(fb, kPageBytes);
              bulk_copy_g2s(sb + L_::kVraw + st * kPageBytes, a.v_pages + off, kPageBytes, fb);
            } else {
              mbar_arrive_expect_tx(fb, kRowDataBytes * kPageTokens + 1024);
              asm volatile(
                  "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                  "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::"r"(sb + L_::kK + st * kKTile),
                  "l"(reinterpret_cast<uint64_t>(&a.tmap)), "r"(0), "r"(0), "r"(0), "r"(cur.h),
                  "r"(pid), "r"(fb)
                  : "memory");
              bulk_copy_g2s(sb + L_::kKsc + st * 1024, a.k_pages + off + kScaleOffset, 512, fb);
              bulk_copy_g2s(sb + L_::kKsc + st * 1024 + 512, a.v_pages + off + kScaleOffset, 512, fb);
            }
          }
        }
        __syncwarp();
        ++k;
        kr.next();
        vr.next();
      }
    }
    // every copy has landed before the CTA ends
    if (lane == 0) {
      const int S = isv ? VS : KS, full = isv ? kVFull : kKFull;
      for (int i = max(0, k - S); i < k; ++i) wait(full + i % S, (i / S) & 1);
    }
  } else if (warp == 1) {
    // ================= S^T = K q^T: one lane
    if (lane == 0) {
      int k = 0;
      Ring<KS> kr;
      Ring<2> sr;
      const uint64_t ad0 = desc(sb + L_::kK, 16, 1024) | ((uint64_t)2 << 61);
      const uint64_t sd0 = desc(sb + L_::kKsc, 16, 128), bd0 = desc(sb + L_::kQ, 128, 1024);
      for_tiles([&](int tile, int, int, int, const Span& sp, int e0, int e1) {
        if (sp.np == 0) return;
        wait(kQFull, tile & 1);
        for (int e = e0; e < e1; ++e, ++k, kr.next(), sr.next()) {
          const int st = kr.slot, b = sr.slot;
          wait(kKFull + st, kr.phase);
          if (k >= 2) wait(kSFree + b, sr.phase ^ 1u);
          if (*s_abort) continue;
          fence_after();
          const uint32_t sfa = tm + T_::kSfa + 4u * b;
          const uint64_t ad = ad0 + st * (kKTile >> 4);
          asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(sfa),
                       "l"(sd0 + st * (1024 >> 4))
                       : "memory");
#pragma unroll
          for (uint32_t part = 0; part < (C::kTwin ? 1 : 2); ++part)
#pragma unroll
            for (uint32_t kb = 0; kb < 4; ++kb)
              asm volatile(
                  "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                  " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, "
                  "%2, %3, [%4], [%5], p;\n}\n" ::"r"(tm + T_::kS + b * C::kScols),
                  "l"(ad + kb * (32 >> 4)), "l"(bd0 + ((part * NR * 128 + kb * 256) >> 4)),
                  "r"(idesc_s<T_::kSfbRows>(kb)), "r"(sfa), "r"(tm + T_::kSfb + part * 4),
                  "r"(part + kb)
                  : "memory");
          commit(bar(kSFull + b));
          commit(bar(kKEmpty + st));
          if (e == e1 - 1) commit(bar(kQEmpty));
        }
      });
      if (k > 0) {  // no MMA in flight when the tensor memory is freed
        commit(bar(kDrain));
        for (uint32_t p = 0; p < kWaitPolls; ++p)
          if (mbar_test(bar(kDrain), 0)) break;
      }
    }
  } else {
    // ================= O^T += V^T P^T: one lane
    if (lane == 0) {
      int k = 0;
      Ring<VB> br;
      const uint64_t ad0 = desc(sb + L_::kV, kVHalf, 1024) | ((uint64_t)2 << 61);
      const uint64_t bd0 = desc(sb + L_::kP, 128, kChunk);
      for_tiles([&](int tile, int, int, int, const Span& sp, int e0, int e1) {
        if (sp.np == 0) return;
        if (tile > 0) wait(kOFree, (tile - 1) & 1);
        for (int e = e0; e < e1; ++e, ++k, br.next()) {
          const int b = br.slot;
          wait(kVReady + b, br.phase);
          wait(kPFull + b, br.phase);
          if (*s_abort) continue;
          fence_after();
          const uint64_t ad = ad0 + b * (kVTile >> 4), bd = bd0 + b * ((NR / 8) * kChunk >> 4);
#pragma unroll
          for (uint32_t ks = 0; ks < 8; ++ks)
            asm volatile(
                "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tm + T_::kO),
                "l"(ad + ks * (2048 >> 4)), "l"(bd + ks * (256 >> 4)), "r"(idesc_o<NR>()),
                "r"((uint32_t)(ks > 0 || e > e0))
                : "memory");
          commit(bar(kPvDone + b));
        }
      });
      if (k > 0) {
        commit(bar(kDrain + 1));
        for (uint32_t p = 0; p < kWaitPolls; ++p)
          if (mbar_test(bar(kDrain + 1), 0)) break;
      }
    }
  }
  } else if (warp >= 4 + 4 * SG) {
    set_regs<kLaunchRegs, C::RD>();
    // ================= q conversion and V dequantisation
    const int t = tid - 32 * (4 + 4 * SG), w = t >> 5;
    const int r8 = lane & 7, blk = ((r8 >> 1) + (lane >> 3)) & 3;  // see below
    int k = 0;
    Ring<VS> vr;
    Ring<VB> br;
    for_tiles([&](int tile, int s, int h, int rt, const Span& sp, int e0, int e1) {
      if (sp.np == 0) return;
      // 16 elements a thread: K-chunk j of row n; the two threads of a 32-block share its
      // largest magnitude.  The rows are on their way while the tile before finishes.
      constexpr int kIt = (NR * 8 + DW * 32 - 1) / (DW * 32);
      uint4 x0[kIt], x1[kIt];
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int n = (t >> 3) + i * DW * 4, row = rt * NR + n, node = row / a.G;
        x0[i] = x1[i] = make_uint4(0u, 0u, 0u, 0u);
        if (n < NR && node < sp.n) {
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (((int64_t)s * a.N + node) * a.H + h * a.G + row % a.G) * kHeadDim +
              16 * (t & 7));
          x0[i] = src[0];
          x1[i] = src[1];
        }
      }
      if (tile > 0) wait(kQEmpty, (tile - 1) & 1);
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int n = (t >> 3) + i * DW * 4, j = t & 7;
        const uint32_t wd[8] = {x0[i].x, x0[i].y, x0[i].z, x0[i].w, x1[i].x, x1[i].y, x1[i].z, x1[i].w};
        float amax = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_float(wd[u] & 0xFFFFu)),
                                   fabsf(bf16_bits_to_float(wd[u] >> 16))));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        const int ef = min(254, (int)(__float_as_uint(amax) >> 23));
        const int E = amax == 0.f ? 0 : max(-122, ef - 127 - 7);
        const float inv = __uint_as_float((uint32_t)(127 - E) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint16_t hc[2], lc[2];
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
                : "=h"(lc[v])
                : "f"((y0 - h0) * 32.f), "f"((y1 - h1) * 32.f));
          }
          hi[u] = (uint32_t)hc[0] | ((uint32_t)hc[1] << 16);
          lo[u] = (uint32_t)lc[0] | ((uint32_t)lc[1] << 16);
        }
        if (n < NR) {
          uint8_t* dst = sm + L_::kQ + (n >> 3) * 1024 + j * 128 + (n & 7) * 16;
          *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + NR * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if ((j & 1) == 0) {
            sm[L_::kSf + n * 4 + (j >> 1)] = (uint8_t)(E + 127);
            sm[L_::kSf + (NR + n) * 4 + (j >> 1)] = (uint8_t)(E + 122);
          }
        }
      }
      fence_async();
      asm volatile("bar.sync 7, %0;\n" ::"n"(32 * DW) : "memory");
      // operand row n's scale word at lane n % 32 of every lane quarter, column n / 32
      if (w < 4) {
#pragma unroll
        for (int part = 0; part < (C::kTwin ? 1 : 2); ++part)
#pragma unroll
          for (int c = 0; c < T_::kSfbW; ++c)
            st1(tm + ((uint32_t)(32 * w) << 16) + T_::kSfb + part * 4 + c,
                *reinterpret_cast<const uint32_t*>(sm + L_::kSf + (part * NR + c * 32 + lane) * 4));
        wait_st();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));

      for (int e = e0; e < e1; ++e, ++k, vr.next(), br.next()) {
        const int st = vr.slot, b = br.slot;
        wait(kVFull + st, vr.phase);
        const int live = s_info[st];
        // Operand row (K index) m holds token 4 (m % 32) + m / 32, the order in which the
        // tensor copy lays out K.  A warp's step: 8 operand rows (r8), lane >> 3 choosing
        // which 32-dim block of each: 16 raw bytes a lane, four 16-byte stores without bank
        // conflicts.  A short loop: the roles' code together must stay near the warps.
        const uint8_t* raw = sm + L_::kVraw + st * kPageBytes;
        if (k >= VB) wait(kPvDone + b, br.phase ^ 1u);
        constexpr int kIts = 16 / DW;
#pragma unroll 1
        for (int it = 0; it < kIts; ++it) {
          const int m = (w * kIts + it) * 8 + r8, tok = 4 * (m & 31) + (m >> 5);
          const uint4 c4 = *reinterpret_cast<const uint4*>(raw + tok * kRowDataBytes + blk * 16);
          const uint32_t sc = raw[kScaleOffset + tok * kRowScaleBytes + blk];
          // 2^(sc - 1), as two factors where it passes bf16's range
          const uint32_t f1 =
              ((tok < live && sc != 255u ? min(sc + 126u, 254u) : 0u) << 7) * 0x10001u;
          const bool big = __any_sync(0xFFFFFFFFu, sc > 128u);
          const uint32_t f2 = ((sc > 128u ? sc - 1u : 127u) << 7) * 0x10001u;
          uint8_t* const dst = sm + L_::kV + b * kVTile + (blk >> 1) * kVHalf + (m >> 3) * 1024 + r8 * 128;
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
            if (big) {
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = bf16_mul2(y[i], f2);
            }
            *reinterpret_cast<uint4*>(dst + ((((blk & 1) * 4 + j) ^ r8) << 4)) =
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
  } else {
    set_regs<kLaunchRegs, C::RS>();
    // ================= softmax: group sg has the rows c0 .. c0 + NC - 1 of a tile
    const int sg = (warp - 4) >> 2, w = warp & 3, t = tid & 127, c0 = sg * NC;
    const uint32_t tl = tm + ((uint32_t)(32 * w) << 16);
    float* const s_nref = reinterpret_cast<float*>(sm + L_::kRef) + c0;
    float* const s_fac = reinterpret_cast<float*>(sm + L_::kFac) + c0;
    float* const s_warp = reinterpret_cast<float*>(sm + L_::kWarp) + 4 * c0;  // [4][NC]
    uint32_t* const s_nan = reinterpret_cast<uint32_t*>(sm + L_::kNan) + c0;
    int* const s_node = reinterpret_cast<int*>(sm + L_::kNode) + c0;
    int* const s_lo = reinterpret_cast<int*>(sm + L_::kLo) + c0;
    uint32_t* const s_mask = reinterpret_cast<uint32_t*>(sm + L_::kMask) + 2 * c0;  // [NC][2]
    auto sync4 = [&]() { asm volatile("bar.sync %0, 128;\n" ::"r"(sg + 1) : "memory"); };
    auto any4 = [&](bool v) {
      uint32_t r;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
          " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(r)
          : "r"((uint32_t)v), "r"(sg + 1)
          : "memory");
      return r != 0u;
    };
    const float cs = a.scale * kLog2e;
    const int tok = 4 * lane + w;  // this lane's token of a page
    int k = 0;
    Ring<KS> kr;
    Ring<2> sr;
    Ring<VB> br;
    for_tiles([&](int tile, int s, int h, int rt, const Span& sp, int e0, int e1) {
      const bool begins = e0 == 0, ends = e1 >= sp.np;
      // ---- the tile's rows
      sync4();  // the tile before is written out
      if (t < NC) {
        const int row = rt * NR + c0 + t, node = row / a.G;
        s_node[t] = node < a.N ? node * a.H + h * a.G + row % a.G : -1;
        uint64_t mk = 0;
        int lo = 0;
        if (node < sp.n) {
          const uint64_t all = sp.n < 64 ? (1ull << sp.n) - 1 : ~0ull;
          auto mask_of = [&](int j) {
            return (a.mask ? a.mask[(int64_t)s * a.N + j] : (2ull << j) - 1) & all;
          };
          auto depth_of = [&](int j) { return max(1, __popcll(mask_of(j))) - 1; };
          mk = mask_of(node);
          if (a.window > 0) {
            const int d = depth_of(node);
            lo = max(0, sp.base + d + 1 - a.window);
            for (int i = 0; i < sp.n; ++i)
              if ((mk >> i) & 1ull) {
                const int di = depth_of(i);
                if (!(di > d - a.window || sp.base + di < a.sinks)) mk &= ~(1ull << i);
              }
          }
        }
        s_mask[2 * t] = (uint32_t)mk;
        s_mask[2 * t + 1] = (uint32_t)(mk >> 32);
        s_lo[t] = lo;
        s_nref[t] = -kUnset;
        s_nan[t] = 0;
      }
      sync4();
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;

      if (sp.np > 0) {
        for (int e = e0; e < e1; ++e, ++k, kr.next(), sr.next(), br.next()) {
          const int st = kr.slot, b = sr.slot, pb = br.slot;
          const int first = page_no(sp, e) * kPageTokens;
          wait(kKFull + st, kr.phase);
          const int live = s_kinfo[st];
          uint32_t vw = *reinterpret_cast<const uint32_t*>(sm + L_::kKsc + st * 1024 + 512 + tok * 4);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kKEmpty + st));
          wait(kSFull + b, sr.phase);
          fence_after();
          // dim blocks of this token's V row that are NaN
          vw = ((vw & 0x7F7F7F7Fu) + 0x01010101u) & vw & 0x80808080u;
          const bool plain = live == kPageTokens && first + kPageTokens <= sp.base &&
                             (a.window == 0 || first > sp.base + 63 - a.window ||
                              first + kPageTokens <= a.sinks);
          // a row sees a draft by its mask, an earlier token from the window's first on;
          // rows without a node see what they like, their results are zeroed
          uint32_t vis = ~0u;
          if (!plain) {
            vis = 0u;
            const int i_g = first + tok, nd = i_g - sp.base;
            if (tok < live) {
#pragma unroll 1
              for (int c = 0; c < NC; ++c) {
                const bool see = nd >= 0 ? ((s_mask[2 * c + ((nd >> 5) & 1)] >> (nd & 31)) & 1u) != 0u
                                         : i_g >= s_lo[c] || i_g < a.sinks;
                vis |= (uint32_t)see << c;
              }
            }
          }
          float x[NC];
          const uint32_t ts = tl + T_::kS + b * C::kScols + c0;
          // S of 16 rows, hi and lo parts added where they are apart
          auto s16 = [&](int c, float* v) {
            ld16(ts + c, v);
            if constexpr (C::kTwin) {
              float y[16];
              ld16(ts + NR + c, y);
              wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += y[i];
            } else {
              wait_ld();
            }
          };
          // -inf where not seen, whatever was computed there
          auto hide16 = [&](int c, float* v) {
            if (plain) return;
            const uint32_t vb = vis >> c;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = (vb >> i) & 1u ? v[i] : -INFINITY;
          };
          for (bool again = false;; again = true) {
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; c += 16) {
              s16(c, x + c);
#pragma unroll
              for (int i = c; i < c + 16; i += 4) {
                const float4 rf = *reinterpret_cast<const float4*>(s_nref + i);
                x[i] = fmaf(x[i], cs, rf.x);
                x[i + 1] = fmaf(x[i + 1], cs, rf.y);
                x[i + 2] = fmaf(x[i + 2], cs, rf.z);
                x[i + 3] = fmaf(x[i + 3], cs, rf.w);
              }
              hide16(c, x + c);
              float m[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) m[i] = fmaxf(x[c + i], x[c + 8 + i]);
#pragma unroll
              for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < o; ++i) m[i] = fmaxf(m[i], m[i + o]);
              top = fmaxf(top, m[0]);
            }
            if (again || !any4(top > kLazy)) break;
            // new references: the page's maximum of each row that has a larger one; what was
            // summed so far is brought to them, and the page's logits are taken once more
#pragma unroll 1
            for (int c = 0; c < NC; c += 16) {
              float v[16];
              s16(c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= cs;
              hide16(c, v);
              const float mx = columns16(v, lane, [](float p, float q) { return fmaxf(p, q); });
              if (lane < 16) s_warp[w * NC + c + lane] = mx;
            }
            if (e > e0) wait(kPvDone + (VB == 1 ? 0 : pb ^ 1), VB == 1 || pb == 0 ? br.phase ^ 1u : br.phase);
            sync4();
            if (t < NC) {
              const float v = fmaxf(fmaxf(s_warp[t], s_warp[NC + t]),
                                    fmaxf(s_warp[2 * NC + t], s_warp[3 * NC + t]));
              const float old = -s_nref[t], now = fmaxf(old, v);
              s_fac[t] = old == kUnset ? 0.f : ex2(old - now);
              s_nref[t] = -now;
            }
            sync4();
#pragma unroll
            for (int c = 0; c < NC; ++c) l[c] *= s_fac[c];
            if (e > e0) {
              fence_after();
#pragma unroll 1
              for (int c = 0; c < NC; c += 16) {
                float o[16];
                ld16(tl + T_::kO + c0 + c, o);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= s_fac[c + i];
                st16(tl + T_::kO + c0 + c, o);
              }
              wait_st();
            }
          }
          // the accumulator has been read: a later page's product may go into it
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSFree + b));
          if (vw != 0u) {
#pragma unroll 1
            for (int c = 0; c < NC; ++c)
              if ((vis >> c) & 1u) atomicOr(s_nan + c, vw);
          }
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            x[c] = ex2(x[c]);
            l[c] += x[c];
          }
          if (k >= VB) wait(kPvDone + pb, br.phase ^ 1u);
          uint8_t* const pd = sm + L_::kP + (pb * (NR / 8) + (c0 >> 3)) * kChunk +
                              (4 * w + (lane >> 3)) * 128 + (lane & 7) * 16;
#pragma unroll
          for (int c = 0; c < NC; c += 8)
            *reinterpret_cast<uint4*>(pd + (c >> 3) * kChunk) =
                make_uint4(pack_bf16(x[c], x[c + 1]), pack_bf16(x[c + 2], x[c + 3]),
                           pack_bf16(x[c + 4], x[c + 5]), pack_bf16(x[c + 6], x[c + 7]));
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kPFull + pb));
        }
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          const float v = columns16(l + c, lane, [](float p, float q) { return p + q; });
          if (lane < 16) s_warp[w * NC + c + lane] = v;
        }
        wait(kPvDone + (VB == 1 ? 0 : br.slot ^ 1), VB == 1 || br.slot == 0 ? br.phase ^ 1u : br.phase);
        sync4();
      } else {
        for (int c = t; c < 4 * NC; c += 128) s_warp[c] = 0.f;
        sync4();
      }
      // ---- the tile's result: this lane's dim of every row
      const bool whole = begins && ends;
      float* const rec = a.rec + (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * (int64_t)(NR * 130);
      if (t < NC) {
        float sum = (s_warp[t] + s_warp[NC + t]) + (s_warp[2 * NC + t] + s_warp[3 * NC + t]);
        if ((rt * NR + c0 + t) / a.G >= sp.n) sum = 0.f;
        const float rf = -s_nref[t];
        if (whole) {
          s_fac[t] = sum == 0.f ? 0.f : 1.f / sum;
          if (a.lse && s_node[t] >= 0)
            a.lse[(int64_t)s * a.N * a.H + s_node[t]] =
                sum == 0.f ? -INFINITY : (log2f(sum) + (rf == kUnset ? 0.f : rf)) * 0.6931471805599453f;
        } else {
          s_fac[t] = sum == 0.f ? 0.f : 1.f;
          rec[NR * 128 + c0 + t] = rf;
          rec[NR * 129 + c0 + t] = sum;
        }
      }
      sync4();
      fence_after();
      // operand position -> dim: the codes of a word were paired i, i + 4
      const int dim = 32 * w + (lane & 24) + ((lane & 1) << 2) + ((lane & 7) >> 1);
      const uint32_t nb = 0x80u << (8 * w);
#pragma unroll 1
      for (int c = 0; c < NC; c += 16) {
        float o[16];
        if (sp.np > 0) {
          ld16(tl + T_::kO + c0 + c, o);
          wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float f = s_fac[c + i];
          const float v = sp.np == 0 || f == 0.f ? 0.f : (s_nan[c + i] & nb) ? NAN : o[i] * f;
          if (whole) {
            const int row = s_node[c + i];
            if (row >= 0)
              a.out[((int64_t)s * a.N * a.H + row) * kHeadDim + dim] =
                  __bfloat16_as_ushort(__float2bfloat16_rn(v));
          } else {
            rec[(c0 + c + i) * 128 + dim] = v;
          }
        }
      }
      fence_before();
      __syncwarp();
      if (sp.np > 0 && lane == 0) mbar_arrive(bar(kOFree));
    });
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
__global__ void __launch_bounds__(128) tree_merge_kernel(const Args a) {
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

template <class C>
cudaError_t launch(Args a, int64_t B, int num_sms, cudaStream_t stream) {
  const int smem = Lay<C>::kBytes;
  auto kern = tree_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // a block that was launched with fewer registers than its roles take would wait for them
  static const int regs = [kern] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs * C::kThreads < C::kRegs) return cudaErrorInvalidConfiguration;
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
// largest.
//               NR SG DW KS VS VB CTAs registers
using C16 = Cfg<16, 1, 8, 2, 3, 1, 2, 40, 104, 56>;
using C32 = Cfg<32, 2, 8, 4, 4, 2, 1, 48, 144, 72>;
using C64 = Cfg<64, 2, 8, 3, 3, 2, 1, 48, 144, 72>;
inline int rows_of(int N, int H, int Hkv) {
  const int rows = N * (H / Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}
inline int ctas_of(int nr) { return nr == 16 ? C16::CTAS : nr == 32 ? C32::CTAS : C64::CTAS; }

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
    case 16: return tree::launch<tree::C16>(a, B, num_sms, stream);
    case 32: return tree::launch<tree::C32>(a, B, num_sms, stream);
    default: return tree::launch<tree::C64>(a, B, num_sms, stream);
  }
}

}  // namespace mx4
