// The steps around tree_paged_decode in a speculative decode step: which drafted
// tokens stand (verify_drafts), the cache rows of the ones that do (accept_rows),
// and sequences that branch and end (fork_pages, free_pages).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace mx4 {

// ---------------------------------------------------------------------------
// verify_drafts.  With p and q the target's and the draft's distributions after node
// `cur`, the children x_1, x_2, ... of cur are tested in order against what is left of p:
//   W_0 = p, T_0 = 1;   x_k stands iff  u T q(x_k) < W(x_k);   else
//   W <- max(W - T q, 0), T <- sum W
// (W / T is the residual distribution; kept unnormalised so nothing is divided), and
// where no child stands the next token is drawn from W by its running sum.
//
// As max(max(p - a, 0) - b, 0) = max(p - a - b, 0) for b >= 0, after k rejections
//   W_k = max(p - S_k q, 0),   S_k = T_0 + ... + T_{k-1}:
// p, q and one number give every residual, none is kept.
//
// W is rounded to 2^-46 of p and then to a multiple of 2^-61, and summed exactly, as integers:
// no order of summation and no cluster size changes a decision.  fp64 and 64-bit shifts and
// conversions run at a small part of fp32's rate here, so the integers are made by fp32
// additions, two values an instruction: adding 3 to a value in [0, 1] leaves its multiple of
// 2^-22 in the sum's low bits, what is left over goes on to smaller constants, and the bits of
// each step are added up as 32-bit integers.  (64-bit integer arithmetic: 73 us for 64 trees
// of 32 nodes over 131072 tokens.)  Sums stop at kFull, just below 2: the test's products and
// the sums themselves have no room for more, and no row of probabilities comes near it.  As
// every partial sum stops there, a row's sum does whatever the order, and is refused.
//
// One cluster of CTAs per sequence, each CTA one contiguous part of the vocabulary, each warp
// one of that.  What the walk looks up (parents, tokens, random numbers, p and q of each draft
// at its parent) is loaded by all threads at once, so accepted drafts cost no dependent loads.
// At a node's first rejection its rows are read, once: a thread keeps E values of p in
// registers and of q in shared memory (a row of 131072 values by eight CTAs, two an SM), and
// every further rejection of a sibling, the sums and the drawing of the next token work on
// those.  E = 0, for vocabularies above 8 x 16384: the rows are read again.  So are those of
// given drafts, whose rejections take one token off the sum: a row is read once, and then the
// 256th of it that the next token is in.
// Every thread runs the walk itself on the same numbers, so it needs no broadcast.
// 64 trees of 32 nodes over 131072 tokens take 65 us (rejections follow one another, about 2 us
// each for a cluster, in two waves of clusters; 77 us over 131073, 104 over 262144 by E = 0), 256
// given chains of 8 over 50001 tokens 30 us (with rows kept by clusters of four half as much
// again), one chain of 4 over 32000 tokens 13 us.  (Rows from memory, an event pair around a graph;
// among other passes on fresh inputs 65, 20 and 9.5 us.)
constexpr int kMaxNodes = 64;
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerUnroll = 8;  // loads in flight per thread and row (E = 0)
constexpr int kVerMaxCluster = 8;

struct VerifyArgs {
  const float* target;
  const float* draft;  // NULL: given drafts
  int64_t t_batch, t_node, d_batch, d_node;  // strides in elements
  const int32_t* tokens;
  const int32_t* parents;
  const float* u_accept;
  const float* u_sample;
  const int32_t* n_nodes;  // NULL: all N
  int N, V;
  int32_t* path;
  int32_t* n_accepted;
  int32_t* next_token;
  uint32_t* status;
};

// (a probability that rounding took above 1 is one)
__device__ __forceinline__ bool prob_ok(float x) { return x >= 0.f && x <= 1.001f; }
// NaN and negative values count as 0 (and what rounding put above 1 as 1)
__device__ __forceinline__ float prob(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
// W values made probabilities; is one no probability?  One comparison each where all lie in
// [0, 1], by their bits.
template <int W>
__device__ __forceinline__ bool clean(float* x) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) most = max(most, __float_as_uint(x[i]));
  bool bad = false;
  if (most > 0x3F800000u) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      bad |= !prob_ok(x[i]);
      x[i] = prob(x[i]);
    }
  }
  return bad;
}

// Two fp32 numbers in one register pair.
using F2 = uint64_t;
__device__ __forceinline__ F2 two(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 two(float a) { return two(a, a); }
__device__ __forceinline__ float first(F2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float second(F2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint32_t bits(F2 x) { return (uint32_t)x + (uint32_t)(x >> 32); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, two(-1.f), a); }

constexpr int64_t kFull = (1ll << 62) - 1;

// S_k as the sum of two fp32 numbers (48 bits)
struct Factor {
  uint64_t sum = 0;  // in units of 2^-56 (S <= 128)
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(uint64_t T) {
    sum += T >> 5;
    const int lz = __clzll((long long)sum);
    const uint64_t m = sum << lz;  // S = m 2^(-56 - lz)
    const float e = __uint_as_float((uint32_t)(127 - 16 - lz) << 23);
    hi = (float)(uint32_t)(m >> 40) * e;
    lo = (float)((uint32_t)(m >> 16) & 0xFFFFFFu) * 0x1p-24f * e;
  }
};

// A sum of n values in units of 2^-61 (at most 64 pairs: the 32-bit sums of the steps' bits).
struct Fixed {
  static constexpr float k1 = 3.f, k2 = 0x1.8p-22f, kc = 0x1.8p-21f, k3 = 0x1.8p-38f;
  uint32_t h = 0, l = 0, lc = 0, z = 0;
  int pairs = 0, corrections = 0;
  // d, each in [0, 1]: multiples of 2^-22, 2^-45 and 2^-61
  __device__ __forceinline__ void put(F2 d) {
    const F2 x = add(d, two(k1)), r = sub(d, add(x, two(-k1)));
    const F2 y = add(r, two(k2)), r2 = sub(r, add(y, two(-k2)));
    h += bits(x);
    l += bits(y);
    z += bits(add(r2, two(k3)));
    ++pairs;
  }
  // c, at most 2^-22 in magnitude: multiples of 2^-44 and 2^-61
  __device__ __forceinline__ void put_small(F2 c) {
    const F2 y = add(c, two(kc)), r = sub(c, add(y, two(-kc)));
    lc += bits(y);
    z += bits(add(r, two(k3)));
    ++corrections;
  }
  // max(p - S q, 0): d + c with d = p - hi q rounded, c its error (exact where d >= 0, the
  // difference of a larger and a smaller number), the product's and lo q
  __device__ __forceinline__ void put(F2 p, F2 q, const Factor& S) {
    const F2 np = mul(two(-S.hi), q), d = add(p, np);
    const F2 c = sub(fma(two(-S.lo), q, add(sub(p, d), np)), fma(two(S.hi), q, np));
    const F2 w = add(d, c);
    const bool a = first(w) > 0.f, b = second(w) > 0.f;
    put(two(a ? first(d) : 0.f, b ? second(d) : 0.f));
    put_small(two(a ? first(c) : 0.f, b ? second(c) : 0.f));
  }
  // (where it is below 4)
  __device__ __forceinline__ int64_t value() const {
    const int n = 2 * pairs, m = 2 * corrections;
    return (int64_t)((uint64_t)coarse() << 39) + ((int64_t)(int)(l - n * 0x34C00000u) << 16) +
           ((int64_t)(int)(lc - m * 0x35400000u) << 17) + (int64_t)(int)(z - (n + m) * 0x2CC00000u);
  }
  // the multiples of 2^-22 alone: they say where 64 bits would not hold the sum
  __device__ __forceinline__ int coarse() const { return (int)(h - 2 * pairs * 0x40400000u); }
  __device__ __forceinline__ int64_t total() const {
    return coarse() >= 3 << 22 ? kFull : min(value(), kFull);
  }
};
__device__ __forceinline__ uint64_t to_fixed(float p) {
  Fixed x;
  x.put(two(p, 0.f));
  return (uint64_t)x.value();
}
__device__ __forceinline__ uint64_t left_of(float p, float q, const Factor& S) {
  Fixed x;
  x.put(two(p, 0.f), two(q, 0.f), S);
  return (uint64_t)x.value();
}

// x >> n, 0 for n of 64 and more
__device__ __forceinline__ uint64_t shift_down(uint64_t x, int n) {
  uint64_t y;
  asm("shr.u64 %0, %1, %2;\n" : "=l"(y) : "l"(x), "r"(n));
  return y;
}
// u in [0, 1) in units of 2^-64
__device__ __forceinline__ uint64_t uniform_fixed(float u) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f));
  return shift_down((uint64_t)(b << 8 | 0x80000000u) << 32, 126 - (int)(b >> 23));
}
// u q < p, exactly: the product's rounding error decides where its rounded value is p
__device__ __forceinline__ bool stands(float u, float q, float p) {
  const float h = u * q;
  return h < p || (h == p && fmaf(u, q, -h) < 0.f);
}

// A sum of numbers of at most kFull, stopped there.  Their top bits, added up alone, say whether
// the 64-bit sum may have wrapped (they alone decide from 3 on).
__device__ __forceinline__ int top(int64_t x) { return (int)(x >> 41); }
__device__ __forceinline__ int64_t stopped(int64_t sum, int tops) {
  return tops >= 3 << 20 ? kFull : min(sum, kFull);
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
  const int tops = __reduce_add_sync(0xFFFFFFFFu, top(x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return stopped(x, tops);
}

template <int E, bool kGiven>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t s = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ float s_row[];  // E > 0: q, value i of thread t at 512 i + t
  __shared__ int32_t s_par[kMaxNodes], s_tok[kMaxNodes], s_path[kMaxNodes];
  __shared__ float s_u[kMaxNodes], s_p[kMaxNodes], s_q[kMaxNodes];
  __shared__ bool s_bad[kMaxNodes];  // p or q of the draft is no probability
  __shared__ int64_t s_warp[2][kVerWarps];       // this CTA's warp sums, of two passes
  __shared__ int64_t s_part[2][kVerMaxCluster];  // the cluster's CTA sums
  __shared__ int64_t s_sub[kVerWarps];
  pdl_launch_dependents();
  pdl_wait();

  int par = -1, tok = 0;
  float u = 0.f;
  if (tid > 0 && tid < a.N) {
    par = a.parents[s * a.N + tid];
    tok = a.tokens[s * a.N + tid];
    u = a.u_accept[s * a.N + tid];
  }
  const float u_next = a.u_sample[s];
  const int n0 = a.n_nodes ? a.n_nodes[s] : a.N, n = min(max(n0, 0), a.N);
  if (n0 != n && rank == 0 && tid == 0) flag(a.status, MX4_STATUS_BAD_LEN);
  if (n < 1) {  // an idle sequence (uniform over the cluster)
    if (rank == 0) {
      if (tid < a.N) a.path[s * a.N + tid] = -1;
      if (tid == 0) {
        a.n_accepted[s] = 0;
        a.next_token[s] = -1;
      }
    }
    return;
  }
  const float* const tgt = a.target + s * a.t_batch;
  const float* const drf = kGiven ? nullptr : a.draft + s * a.d_batch;
  // The cluster's other CTAs run once they have arrived here: their shared memory may be
  // written after the wait that goes with it, in front of the first sum.
  cluster.barrier_arrive();
  if (tid < kMaxNodes) {
    if (tid >= n) {
      par = -1;
    } else if (par != -1 && (par < 0 || par >= tid || tok < 0 || tok >= a.V)) {
      flag(a.status, MX4_STATUS_BAD_INDEX);
      par = -1;  // never tested
    }
    s_par[tid] = par;
    s_tok[tid] = tok;
    s_path[tid] = tid == 0 ? 0 : -1;
    s_u[tid] = u;
    const float p = par >= 0 ? tgt[par * a.t_node + tok] : 0.f;
    const float q = kGiven ? 1.f : par >= 0 ? drf[par * a.d_node + tok] : 0.f;
    s_p[tid] = prob(p);
    s_q[tid] = prob(q);
    s_bad[tid] = !prob_ok(p) || !prob_ok(q);
  }
  __syncthreads();

  // this CTA's part of the vocabulary, and this warp's part of that
  // (V <= 2^24; C is a power of two)
  const int log2c = 31 - __clz(C);
  auto cta_begin = [&](int r) { return a.V * r >> log2c; };
  const int c0 = cta_begin(rank), c1 = cta_begin(rank + 1);
  auto warp_begin = [&](int w) { return c0 + (c1 - c0) * w / kVerWarps; };
  const int v0 = warp_begin(warp), v1 = warp_begin(warp + 1);
  bool bad = false;

  int cur = 0, k = 0;  // the node; its children rejected so far
  Factor S;
  uint64_t gone = 0;   // (given drafts) those, by node
  const float* p_row = tgt;
  const float* q_row = drf;
  // E > 0: values v0 + 32 i + lane of p
  float f[E > 0 ? E : 1];
  bool loaded = false;
  auto load = [&](bool with_q) {
    const int left = v1 - v0 - lane;  // values from this lane's first on
    if (with_q) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(
                         smem_addr(s_row + kVerThreads * i + tid)),
                     "l"(32 * i < left ? q_row + v0 + lane + 32 * i : q_row),
                     "r"(32 * i < left ? 4 : 0)
                     : "memory");
    }
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = 32 * i < left ? __ldg(p_row + v0 + lane + 32 * i) : 0.f;
    bad |= clean<E>(f);
    if (with_q) {
      asm volatile("cp.async.wait_all;\n" ::: "memory");
#pragma unroll 8
      for (int i = 0; i < E; ++i) {  // (a thread's own values: no barrier)
        const float q = s_row[kVerThreads * i + tid];
        bad |= !prob_ok(q);
        s_row[kVerThreads * i + tid] = prob(q);
      }
    }
    loaded = true;
  };
  // what is left of token v
  auto at_mem = [&](int v, float pv, float qv) -> uint64_t {
    if (!kGiven) return k == 0 ? to_fixed(pv) : left_of(pv, qv, S);
    for (uint64_t g = gone; g; g &= g - 1)
      if (s_tok[__ffsll((long long)g) - 1] == v) return 0;
    return to_fixed(pv);
  };
  // its sum over b0 <= v < b1 by one warp (all lanes get it)
  auto range_sum = [&](int b0, int b1) {
    int64_t sum = 0;
    const bool two_rows = !kGiven && k > 0;
    Fixed x;
    for (int b = b0 + lane; b < b1; b += 32 * kVerUnroll) {
      float pv[kVerUnroll], qv[kVerUnroll];
#pragma unroll
      for (int i = 0; i < kVerUnroll; ++i) {
        const int v = b + 32 * i;
        pv[i] = v < b1 ? p_row[v] : 0.f;
        qv[i] = two_rows && v < b1 ? q_row[v] : 0.f;
      }
      bad |= clean<kVerUnroll>(pv);
      if (two_rows) bad |= clean<kVerUnroll>(qv);
      if (kGiven)
        for (uint64_t g = gone; g; g &= g - 1) {
          const int at = s_tok[__ffsll((long long)g) - 1] - b;
#pragma unroll
          for (int i = 0; i < kVerUnroll; ++i)
            if (at == 32 * i) pv[i] = 0.f;
        }
#pragma unroll
      for (int i = 0; i < kVerUnroll; i += 2) {
        if (two_rows)
          x.put(two(pv[i], pv[i + 1]), two(qv[i], qv[i + 1]), S);
        else
          x.put(two(pv[i], pv[i + 1]));
      }
      if (x.pairs >= 64) {
        sum = min(sum + x.total(), kFull);
        x = Fixed{};
      }
    }
    return warp_sum(min(sum + x.total(), kFull));
  };
  // the sum of the residual, with the warp and CTA sums left in place `pass & 1`
  int pass = 0;
  auto total = [&]() -> uint64_t {
    int64_t ws = 0;
    if constexpr (E > 0) {
      Fixed x;
      if (k == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 2) x.put(two(f[i], f[i + 1]));
      } else {
#pragma unroll
        for (int i = 0; i < E; i += 2)
          x.put(two(f[i], f[i + 1]),
                two(s_row[kVerThreads * i + tid], s_row[kVerThreads * (i + 1) + tid]), S);
      }
      ws = x.total();
      ws = warp_sum(ws);
    } else {
      ws = range_sum(v0, v1);
    }
    if (pass == 0) cluster.barrier_wait();
    ++pass;
    // (the places two passes back have been read by all before the barrier of the last pass)
    if (lane == 0) s_warp[pass & 1][warp] = ws;
    __syncthreads();
    if (warp == 0) {
      const int64_t cs = warp_sum(lane < kVerWarps ? s_warp[pass & 1][lane] : 0);
      if (lane < C) *cluster.map_shared_rank(&s_part[pass & 1][rank], lane) = cs;
    }
    cluster.sync();
    int64_t t = 0;
    int tops = 0;
#pragma unroll
    for (int i = 0; i < kVerMaxCluster; ++i) {
      const int64_t x = i < C ? s_part[pass & 1][i] : 0;
      t += x;
      tops += top(x);
    }
    return (uint64_t)max(stopped(t, tops), (int64_t)0);
  };

  // children of cur, by node (they come after it)
  auto children = [&]() {
    return (uint64_t)__ballot_sync(0xFFFFFFFFu, s_par[lane] == cur) |
           (uint64_t)__ballot_sync(0xFFFFFFFFu, s_par[32 + lane] == cur) << 32;
  };
  int acc = 1;
  bool summed = false;  // the last pass is of the present residual
  uint64_t T = 1ull << 61;
  for (uint64_t kids = children(); kids;) {
    const int j = __ffsll((long long)kids) - 1;
    kids &= kids - 1;
    const float pv = s_p[j], qv = s_q[j];
    bad |= s_bad[j];
    uint64_t w = 0;  // what is left of its token
    bool ok;
    if constexpr (kGiven) {
      w = at_mem(s_tok[j], pv, 0.f);
      ok = k == 0 ? s_u[j] < pv : __umul64hi(uniform_fixed(s_u[j]), T) < w;
    } else {
      // floor(u T q) < W, both integers, T q rounded down to one
      ok = k == 0 ? stands(s_u[j], qv, pv)
                  : __umul64hi(uniform_fixed(s_u[j]), __umul64hi(T << 2, to_fixed(qv) << 1)) <
                        left_of(pv, qv, S);
    }
    if (ok) {
      cur = j;
      p_row = tgt + (int64_t)j * a.t_node;
      if constexpr (!kGiven) q_row = drf + (int64_t)j * a.d_node;
      S = Factor{};
      T = 1ull << 61;
      k = 0;
      gone = 0;
      summed = loaded = false;
      if (tid == 0) s_path[acc] = j;
      ++acc;
      kids = children();
      continue;
    }
    if (E > 0 && !loaded) load(true);
    if constexpr (kGiven) {
      // the row is summed once; what has been rejected is taken off that sum, and in the end
      // off the CTA's and the warp's that hold it
      if (k == 0) T = total();
      if (T < kFull) T -= w;
      summed = true;
      if (w != 0) gone |= 1ull << j;  // (a token once)
      ++k;
    } else {
      S.add(T);
      ++k;
      T = total();
      summed = true;
    }
    if (T >= kFull) break;  // no probabilities
    if (T == 0) {  // nothing left (p <= q everywhere): draw from p itself
      k = 0;
      gone = 0;
      summed = loaded = false;
      break;
    }
  }
  if (!summed) {
    if (E > 0 && !loaded) load(false);
    T = total();
  }

  // of a sum over b0 <= v < b1, less what has been rejected there
  auto kept = [&](uint64_t sum, int b0, int b1) -> uint64_t {
    if (kGiven)
      for (uint64_t g = gone; g; g &= g - 1) {
        const int j = __ffsll((long long)g) - 1;
        if (s_tok[j] >= b0 && s_tok[j] < b1) sum -= to_fixed(s_p[j]);
      }
    return sum;
  };
  // the next token: the first v whose running sum exceeds u T
  const uint64_t left = __umul64hi(uniform_fixed(u_next), T);
  // the first lane whose running sum of x exceeds `left` (-1: none); `before` goes on to it
  uint64_t before = 0;
  auto scan = [&](uint64_t x) {
    uint64_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    const int l = __ffs(__ballot_sync(0xFFFFFFFFu, before + inc > left)) - 1;
    before += __shfl_sync(0xFFFFFFFFu, l < 0 ? inc : inc - x, l < 0 ? 31 : l);
    return l;
  };
  int at = scan(lane < C ? kept(s_part[pass & 1][lane & (kVerMaxCluster - 1)], cta_begin(lane),
                                cta_begin(lane + 1)) : 0);  // the CTA
  if (T == 0 || T >= kFull) at = -1;  // a row of zeros, or of 2 or more: no token
  if (at == rank) {
    // (one is always found)
    const int w = scan(lane < kVerWarps ? kept(s_warp[pass & 1][lane & (kVerWarps - 1)],
                                               warp_begin(lane), warp_begin(lane + 1)) : 0) &
                  (kVerWarps - 1);
    // the warp's part in sixteenths, then one warp's sixteenth 32 values at a time (from the L2
    // cache: every thread's own values, by code for each of them, would be 90 KB of it)
    const int w0 = warp_begin(w), w1 = warp_begin(w + 1);
    auto part = [&](int i) { return w0 + (w1 - w0) * i / kVerWarps; };
    const uint64_t sum = range_sum(part(warp), part(warp + 1));
    if (lane == 0) s_sub[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const int i = scan(lane < kVerWarps ? s_sub[lane & (kVerWarps - 1)] : 0) & (kVerWarps - 1);
      const int end = part(i + 1);
      const bool two_rows = !kGiven && k > 0;
      int found = end - 1, l = -1;
#pragma unroll 1
      for (int b = part(i); b < end && l < 0; b += 32 * kVerUnroll) {
        float pv[kVerUnroll], qv[kVerUnroll];
#pragma unroll
        for (int r = 0; r < kVerUnroll; ++r) {
          const int v = b + 32 * r + lane;
          pv[r] = v < end ? p_row[v] : 0.f;
          qv[r] = two_rows && v < end ? q_row[v] : 0.f;
        }
#pragma unroll 1
        for (int r = 0; r < kVerUnroll && l < 0; ++r) {
          l = scan(at_mem(b + 32 * r + lane, prob(pv[0]), prob(qv[0])));
          if (l >= 0) found = min(b + 32 * r + l, found);
#pragma unroll
          for (int j = 0; j + 1 < kVerUnroll; ++j) {
            pv[j] = pv[j + 1];
            qv[j] = qv[j + 1];
          }
        }
      }
      if (lane == 0) a.next_token[s] = found;
    }
  }
  if (rank == 0) {
    if (at < 0 && tid == 0) {
      a.next_token[s] = -1;
      flag(a.status, MX4_STATUS_BAD_VALUE);
    }
    if (tid == 0) a.n_accepted[s] = acc;
    __syncthreads();
    if (tid < a.N) a.path[s * a.N + tid] = s_path[tid];
  }
  if (bad) flag(a.status, MX4_STATUS_BAD_VALUE);
}

template <int E>
cudaError_t launch_verify_e(const VerifyArgs& a, cudaLaunchConfig_t& cfg) {
  cfg.dynamicSmemBytes = E * kVerThreads * sizeof(float);
  if (cfg.dynamicSmemBytes > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(verify_kernel<E, false>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, verify_kernel<E, false>, a);
}

cudaError_t launch_verify(const float* target, const float* draft, const int64_t* strides,
                          const int32_t* tokens, const int32_t* parents, const float* u_accept,
                          const float* u_sample, const int32_t* n_nodes, int64_t B, int N, int V,
                          int32_t* path, int32_t* n_accepted, int32_t* next_token,
                          uint32_t* status, int num_sms, cudaStream_t stream) {
  VerifyArgs a{target, draft, strides[0], strides[1], strides[2], strides[3], tokens, parents,
               u_accept, u_sample, n_nodes, N, V, path, n_accepted, next_token, status};
  // CTAs a sequence: few (an exchange costs the more), but enough that a thread keeps at most
  // 32 values (of rows that are kept), and that a small batch takes about two CTAs an SM of 2048
  // values or more
  int C = 1;
  while (C < kVerMaxCluster && ((draft && V > (int64_t)C * kVerThreads * 32) ||
                                (B * C * 2 <= 2 * (int64_t)num_sms && V / C > 4096)))
    C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * C));
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // the largest part of a warp, in rows of 32 values
  const int part = ((V + C - 1) / C + kVerWarps - 1) / kVerWarps, rows = (part + 31) / 32;
  if (!draft) return cudaLaunchKernelEx(&cfg, verify_kernel<0, true>, a);
  if (rows > 32) return launch_verify_e<0>(a, cfg);
  if (rows > 16) return launch_verify_e<32>(a, cfg);
  if (rows > 8) return launch_verify_e<16>(a, cfg);
  return launch_verify_e<8>(a, cfg);
}

// ---------------------------------------------------------------------------
// Cache rows.  A pool is MXFP4 (64 data bytes and 4 scale bytes a row, head after head)
// or the fp8 index pool (128 data bytes a row, no scales).
struct Pools {
  uint8_t* k;
  uint8_t* v;
  int64_t kv_page, kv_head;
  uint8_t* idx;  // NULL: none
  int64_t idx_page;
  int idx_fp8;
  int Hkv;
  int64_t num_pages;
  __host__ __device__ int parts() const { return 2 * Hkv + (idx ? 1 : 0); }
  // Part r of page p (K heads, V heads, the index key) and whether it is an fp8 one.
  __device__ uint8_t* part(int r, int64_t p, bool& fp8) const {
    fp8 = r == 2 * Hkv && idx_fp8;
    if (r < Hkv) return k + p * kv_page + r * kv_head;
    if (r < 2 * Hkv) return v + p * kv_page + (r - Hkv) * kv_head;
    return idx + p * idx_page;
  }
};

// accept_rows: the rows of the accepted nodes move to the sequence's first draft rows.
// One CTA per (sequence, part).  Rows move towards lower places (path[i] >= i), so a
// row's new place may be another's old one: every row is read into registers before
// any is written.  16 bytes a thread and row piece, at most 8 pieces a row.  A few dependent
// loads and a launch: 9 us alone, 17 us for 256 trees of 64 nodes with 8 KV heads.
constexpr int kAccThreads = 256;
__global__ void __launch_bounds__(kAccThreads)
accept_kernel(const int32_t* __restrict__ path, const int32_t* __restrict__ n_accepted,
              const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ n_nodes, int N,
              const int32_t* __restrict__ table, int64_t bt_width, Pools pools,
              int32_t* __restrict__ new_lens, uint32_t* status) {
  __shared__ int64_t s_src[kMaxNodes], s_dst[kMaxNodes];  // page * 128 + row; -1: stays
  pdl_wait();
  const int64_t s = blockIdx.x;
  const int r = blockIdx.y, tid = threadIdx.x;
  const int n = n_nodes ? n_nodes[s] : N;
  const int64_t L = seq_lens[s];
  const int acc = n_accepted[s];
  bool ok = n >= 0 && n <= N && L >= n && L <= bt_width * kPageTokens && acc >= 0 && acc <= n;
  const bool len_ok = ok;
  const int64_t base = L - n;
  int bad_page = 0;
  if (ok && tid < kMaxNodes) {
    int64_t src = -1, dst = -1;
    if (tid < acc) {
      const int32_t p = path[s * N + tid];
      const int32_t prev = tid > 0 ? path[s * N + tid - 1] : -1;
      if (p <= prev || p >= n) {
        ok = false;
      } else {  // (a row that stays has to be on a page as well)
        const int64_t i = base + p, o = base + tid;
        const int32_t sp = table[s * bt_width + i / kPageTokens];
        const int32_t dp = table[s * bt_width + o / kPageTokens];
        if (sp < 0 || sp >= pools.num_pages || dp < 0 || dp >= pools.num_pages) {
          bad_page = 1;
          ok = false;
        } else if (p > tid) {
          src = (int64_t)sp * kPageTokens + i % kPageTokens;
          dst = (int64_t)dp * kPageTokens + o % kPageTokens;
        }
      }
    }
    s_src[tid] = src;
    s_dst[tid] = dst;
  }
  bad_page = __syncthreads_or(bad_page);
  if (!__syncthreads_and(ok)) {  // the sequence is left as it is
    if (r == 0 && tid == 0) {
      flag(status, !len_ok ? MX4_STATUS_BAD_LEN : bad_page ? MX4_STATUS_BAD_PAGE
                                                           : MX4_STATUS_BAD_INDEX);
      new_lens[s] = (int32_t)L;
    }
    return;
  }
  if (r == 0 && tid == 0) new_lens[s] = (int32_t)(base + acc);
  if (acc == 0) return;
  // pieces: 8 a row of an fp8 part; of an MXFP4 part 4 of data and 1 of scales
  uint4 x[2];
  bool fp8;
  pools.part(r, 0, fp8);
  const int per = fp8 ? 8 : 5;
  auto at = [&](int64_t slot, int piece) -> uint8_t* {
    bool f;
    uint8_t* b = pools.part(r, slot / kPageTokens, f);
    const int row = (int)(slot % kPageTokens);
    if (f) return b + row * 128 + piece * 16;
    return piece < 4 ? b + row * kRowDataBytes + piece * 16
                     : b + kScaleOffset + row * kRowScaleBytes;
  };
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = tid + u * kAccThreads, i = e / per, piece = e % per;
    if (i < acc && s_src[i] >= 0) {
      if (!fp8 && piece == 4)
        x[u].x = *reinterpret_cast<const uint32_t*>(at(s_src[i], piece));
      else
        x[u] = *reinterpret_cast<const uint4*>(at(s_src[i], piece));
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = tid + u * kAccThreads, i = e / per, piece = e % per;
    if (i < acc && s_src[i] >= 0) {
      if (!fp8 && piece == 4)
        *reinterpret_cast<uint32_t*>(at(s_dst[i], piece)) = x[u].x;
      else
        *reinterpret_cast<uint4*>(at(s_dst[i], piece)) = x[u];
    }
  }
}
static_assert(2 * kAccThreads >= 8 * kMaxNodes, "a CTA's pieces");

cudaError_t launch_accept(const int32_t* path, const int32_t* n_accepted, const int32_t* seq_lens,
                          const int32_t* n_nodes, int64_t B, int N, const int32_t* table,
                          int64_t bt_width, uint8_t* k, uint8_t* v, int64_t kv_page,
                          int64_t kv_head, int Hkv, uint8_t* idx, int64_t idx_page, int idx_fp8,
                          int64_t num_pages, int32_t* new_lens, uint32_t* status,
                          cudaStream_t stream) {
  const Pools pools{k, v, kv_page, kv_head, idx, idx_page, idx_fp8, Hkv, num_pages};
  return launch_pdl(accept_kernel, dim3((unsigned)B, (unsigned)pools.parts()), dim3(kAccThreads),
                    0, stream, path, n_accepted, seq_lens, n_nodes, N, table, bt_width, pools,
                    new_lens, status);
}

// ---------------------------------------------------------------------------
// fork_pages and free_pages.  Free page ids are a stack: free_list[0 .. free_count).
//
// fork: a child of table row r shares the full pages of r (one more reference each); its
// partly filled last page is a page popped off the stack, with the used rows copied.
// Child i's page is the one under those of the children before it, found by a running
// count, so the outcome does not depend on scheduling.
// Two kernels: one CTA does the counting and the popping (a serial dependence over the
// children, of 4 bytes each); then one CTA per (child, part) copies rows, the first
// part's CTA also the table row and the references.  With the free after it, 512 children of
// 64 sequences with 8 KV heads take 28 us (10 us of them the copies at HBM's rate), four
// children of one 17 us: launches.
constexpr int kForkThreads = 1024;
__global__ void __launch_bounds__(kForkThreads)
fork_assign_kernel(const int32_t* __restrict__ rows, int64_t n, int64_t B, int64_t bt_width,
                   const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ free_list,
                   int32_t* free_count, int64_t num_pages, int32_t* __restrict__ child,
                   int32_t* __restrict__ child_lens, uint32_t* status) {
  __shared__ int s_warp[32];
  __shared__ int s_taken;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int have = (int)min((int64_t)max(*free_count, 0), num_pages);
  if (tid == 0) s_taken = 0;
  __syncthreads();
  for (int64_t b = 0; b < n; b += kForkThreads) {
    const int64_t i = b + tid;
    int need = 0, L = 0;
    if (i < n) {
      const int r = rows[i];
      if (r < 0 || r >= B) {
        flag(status, MX4_STATUS_BAD_INDEX);
      } else {
        L = seq_lens[r];
        if (L < 0 || L > bt_width * kPageTokens) {
          flag(status, MX4_STATUS_BAD_LEN);
          L = 0;
        }
      }
      need = L % kPageTokens != 0;
    }
    int inc = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = s_taken;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    const int rank = before + inc - need;
    if (i < n) {
      if (need) {
        int32_t page = rank < have ? free_list[have - 1 - rank] : -1;
        if (page < 0 || page >= num_pages) {
          flag(status, rank < have ? MX4_STATUS_BAD_PAGE : MX4_STATUS_NO_PAGES);
          page = -1;
          L = 0;  // no page: no child
        }
        child[i * bt_width + (L / kPageTokens)] = page;
      }
      child_lens[i] = L;
    }
    __syncthreads();
    if (tid == kForkThreads - 1) s_taken = before + inc;
    __syncthreads();
  }
  if (tid == 0) *free_count = have - min(s_taken, have);
}

constexpr int kCopyThreads = 128;
__global__ void __launch_bounds__(kCopyThreads)
fork_copy_kernel(const int32_t* __restrict__ rows, int64_t n, int64_t bt_width,
                 const int32_t* __restrict__ table, int32_t* refs, Pools pools,
                 int32_t* __restrict__ child, const int32_t* __restrict__ child_lens,
                 uint32_t* status) {
  pdl_wait();
  const int64_t i = blockIdx.x;
  const int r = blockIdx.y, tid = threadIdx.x;
  const int L = child_lens[i];
  const int full = L / kPageTokens, rem = L % kPageTokens;
  const int32_t* src_row = table + (int64_t)(L > 0 ? rows[i] : 0) * bt_width;
  int32_t* const row = child + i * bt_width;
  if (r == 0) {
    for (int64_t j = tid; j < bt_width; j += kCopyThreads) {
      if (j < full) {
        const int32_t p = src_row[j];
        row[j] = p;
        if (p >= 0 && p < pools.num_pages)
          atomicAdd(refs + p, 1);
        else
          flag(status, MX4_STATUS_BAD_PAGE);
      } else if (j > full || rem == 0) {
        row[j] = -1;
      } else {
        refs[row[j]] = 1;  // the popped page
      }
    }
  }
  if (rem == 0) return;
  const int32_t sp = src_row[full], dp = row[full];
  if (sp < 0 || sp >= pools.num_pages) {
    if (r == 0 && tid == 0) flag(status, MX4_STATUS_BAD_PAGE);
    return;
  }
  bool fp8;
  const uint8_t* from = pools.part(r, sp, fp8);
  uint8_t* to = pools.part(r, dp, fp8);
  // four 16-byte pieces a thread (all of an MXFP4 part) and its scale word, all loaded before
  // the first is stored
  const int pieces = rem * (fp8 ? 8 : 4);
  uint32_t sc = 0;
  if (!fp8 && tid < rem) sc = reinterpret_cast<const uint32_t*>(from + kScaleOffset)[tid];
  for (int b = 0; b < pieces; b += 4 * kCopyThreads) {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i * kCopyThreads + tid < pieces)
        x[i] = reinterpret_cast<const uint4*>(from)[b + i * kCopyThreads + tid];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i * kCopyThreads + tid < pieces)
        reinterpret_cast<uint4*>(to)[b + i * kCopyThreads + tid] = x[i];
  }
  if (!fp8 && tid < rem) reinterpret_cast<uint32_t*>(to + kScaleOffset)[tid] = sc;
}
static_assert(kCopyThreads >= kPageTokens, "a thread a scale word");

cudaError_t launch_fork(const int32_t* rows, int64_t n, const int32_t* table, int64_t B,
                        int64_t bt_width, const int32_t* seq_lens, int32_t* refs,
                        const int32_t* free_list, int32_t* free_count, uint8_t* k, uint8_t* v,
                        int64_t kv_page, int64_t kv_head, int Hkv, uint8_t* idx,
                        int64_t idx_page, int idx_fp8, int64_t num_pages, int32_t* child,
                        int32_t* child_lens, uint32_t* status, cudaStream_t stream) {
  const Pools pools{k, v, kv_page, kv_head, idx, idx_page, idx_fp8, Hkv, num_pages};
  cudaError_t e = launch_pdl(fork_assign_kernel, dim3(1), dim3(kForkThreads), 0, stream, rows, n,
                             B, bt_width, seq_lens, free_list, free_count, num_pages, child,
                             child_lens, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_copy_kernel, dim3((unsigned)n, (unsigned)pools.parts()),
                    dim3(kCopyThreads), 0, stream, rows, n, bt_width, table, refs, pools, child,
                    (const int32_t*)child_lens, status);
}

// free: one reference less for every page of the rows; a page whose count reaches 0 goes
// back on the stack, ascending by id (whatever order the references went in).  The one
// decrement that takes a count from 1 to 0 marks the page by -1 in its place; a second
// kernel, one CTA, turns the marks into 0 and pushes them by a running count over the
// ids: 4 bytes a page of the pool.
constexpr int kFreeThreads = 256;
constexpr int kFreed = -1;

// One reference less for the page of entry j of row s.
__device__ __forceinline__ void free_entry(const int32_t* __restrict__ table, int64_t s,
                                           int64_t bt_width, int64_t j, int32_t* refs,
                                           int64_t num_pages, uint32_t* status) {
  const int32_t p = table[s * bt_width + j];
  if (p < 0 || p >= num_pages) {
    flag(status, MX4_STATUS_BAD_PAGE);
    return;
  }
  int32_t c = *reinterpret_cast<volatile int32_t*>(refs + p);
  for (;;) {  // ends: every failed exchange is another thread's success
    if (c <= 0) {  // a page that nobody holds (or that this call has already freed)
      flag(status, MX4_STATUS_BAD_REF);
      return;
    }
    const int32_t seen = atomicCAS(refs + p, c, c == 1 ? kFreed : c - 1);
    if (seen == c) return;
    c = seen;
  }
}

// The pages of row s, or -1 for a bad length.
__device__ __forceinline__ int64_t free_pages_of(const int32_t* __restrict__ lens, int64_t s,
                                                 int64_t bt_width) {
  const int64_t L = lens[s];
  return L < 0 || L > bt_width * kPageTokens ? -1 : (L + kPageTokens - 1) / kPageTokens;
}

__global__ void __launch_bounds__(kFreeThreads)
free_refs_kernel(const int32_t* __restrict__ table, int64_t n, int64_t bt_width,
                 const int32_t* __restrict__ lens, int32_t* refs, int64_t num_pages,
                 uint32_t* status) {
  pdl_wait();
  const int64_t s = blockIdx.x, pages = free_pages_of(lens, s, bt_width);
  if (pages < 0 && threadIdx.x == 0) flag(status, MX4_STATUS_BAD_LEN);
  for (int64_t j = threadIdx.x; j < pages; j += kFreeThreads)
    free_entry(table, s, bt_width, j, refs, num_pages, status);
}

// kAll: the references too, of few rows, by the same CTA (a warp a row): one launch instead of
// two.
template <bool kAll>
__global__ void __launch_bounds__(kForkThreads)
free_push_kernel(const int32_t* __restrict__ table, int64_t n, int64_t bt_width,
                 const int32_t* __restrict__ lens, int32_t* refs, int64_t num_pages,
                 int32_t* __restrict__ free_list, int32_t* free_count, uint32_t* status) {
  __shared__ int s_warp[32];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if constexpr (kAll) {
    for (int64_t s = warp; s < n; s += kForkThreads / 32) {
      const int64_t pages = free_pages_of(lens, s, bt_width);
      if (pages < 0 && lane == 0) flag(status, MX4_STATUS_BAD_LEN);
      for (int64_t j = lane; j < pages; j += 32)
        free_entry(table, s, bt_width, j, refs, num_pages, status);
    }
    __threadfence_block();
    __syncthreads();
  }
  int64_t top = max(*free_count, 0);
  constexpr int E = 8;  // ids a thread and round
  for (int64_t b = 0; b < num_pages; b += (int64_t)kForkThreads * E) {
    const int64_t p0 = b + (int64_t)tid * E;
    uint32_t mine = 0;
    int32_t c[E];
    // (past the L1, where the references' atomics are)
#pragma unroll
    for (int e = 0; e < E; ++e) c[e] = p0 + e < num_pages ? __ldcg(refs + p0 + e) : 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c[e] == kFreed) mine |= 1u << e;
    int inc = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    int64_t to = top + before + inc - __popc(mine);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((mine >> e) & 1u) {
        refs[p0 + e] = 0;
        if (to < num_pages)
          free_list[to] = (int32_t)(p0 + e);
        else
          flag(status, MX4_STATUS_BAD_REF);  // more free pages than pages
        ++to;
      }
    top += all;
    __syncthreads();
  }
  if (tid == 0) *free_count = (int32_t)min(top, num_pages);
}

// Up to this many table entries one CTA takes the references as well.
constexpr int64_t kFreeSmall = 4096;

cudaError_t launch_free(const int32_t* table, int64_t n, int64_t bt_width, const int32_t* lens,
                        int32_t* refs, int64_t num_pages, int32_t* free_list,
                        int32_t* free_count, uint32_t* status, cudaStream_t stream) {
  if (n * bt_width <= kFreeSmall)
    return launch_pdl(free_push_kernel<true>, dim3(1), dim3(kForkThreads), 0, stream, table, n,
                      bt_width, lens, refs, num_pages, free_list, free_count, status);
  cudaError_t e = launch_pdl(free_refs_kernel, dim3((unsigned)n), dim3(kFreeThreads), 0, stream,
                             table, n, bt_width, lens, refs, num_pages, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(free_push_kernel<false>, dim3(1), dim3(kForkThreads), 0, stream, table, n,
                    bt_width, lens, refs, num_pages, free_list, free_count, status);
}

}  // namespace mx4
