// ops_attn.cu -- the attention operators of include/m3_ops.h.
//
//   attn_tc_kernel   tcgen05: 2 x 128 query rows of one KV head against a run
//                    of 128-key tiles; packed prompts (causal) or a shared
//                    prefix in pages (partial results)
//   attn_own_kernel  warp MMA: one row's query heads against its own pages
//   attn_join_kernel joins the partial results of a row by log-sum-exp (few
//                    positions: the own kernel's CTAs do, as a cluster)
#include <cudaTypedefs.h>
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <mutex>
#include <string>

#include "attention.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "m3_ops.h"
#include "ops.cuh"

namespace m3 {

namespace {

__device__ int g_ops_err;  // first error word of this file's kernels (m3_ops_sync_status)

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {  // two fp32 lanes
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float ex2(float x) {  // 2^x, one MUFU instruction; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ----------------------------------------------------- tcgen05 attention ---
// Rows are (query token, query head of the group): the heads that share a KV
// head sit side by side in one tile, so a K/V tile is read once for all of
// them and a causal tile of 128 rows spans few tokens.
//
// One CTA: warp 0 brings Q and the K/V tiles by TMA, warps 1 and 2 issue the
// MMAs of row tiles 0 and 1, warps 4..7 and 8..11 are their softmax with one row per thread (a TMEM lane is a row: no shuffles).  S = Q K^T goes to
// tensor memory; the softmax reads it, writes P (16 bit) over it and the next
// MMA takes P from there, O += P V, also in tensor memory.  The two row
// tiles alternate: while one's softmax runs, the other's products do.
//
// The running maximum is raised, and O rescaled, only when a row's maximum
// has grown by more than 2^8 since (P then stays below 2^8, and sums and
// products are relative to the same reference, so nothing is lost).
//
// What bounds it: a key tile of both row tiles is 2048 cycles of products and as
// many of exponentials, and takes about 3300: a row tile's softmax (1850) and
// then the rest of its O += P V, the next S and the hand-overs (1430), the other
// row tile's in between.  2 x 9000 tokens, 32 heads on 8, D 128, bf16: 1.29 ms,
// 1030 TFLOP/s, under the power cap that a run of seconds meets; 1.10 ms, 1200
// TFLOP/s, in runs too short for it (tensor pipe and MUFU each 56 % active under
// the profiler).  Short prompts are bound by a CTA's own length, about 9 us for three key tiles, of
// which 5 are its beginning and end (code that runs once is fetched then).
constexpr int kTile = 128;           // rows of a row tile, keys of a key tile
constexpr float kRaise = 8.0f;       // log2 units

// NT row tiles.  Two are for whole SMs of work.  With one the CTA leaves room
// for another kernel's beside it (m3_attn_prefix: a CTA of attn_own_kernel) and
// a call of few rows spreads over twice as many SMs.
template <int D, int NT>
struct TcShape {
  static constexpr int threads = 128 + 128 * NT;
  static constexpr int columns = 256 * NT;                // of tensor memory: S, then O
  static constexpr uint32_t tile_bytes = kTile * D * 2;  // Q, K and V tiles alike
  static constexpr uint32_t half_bytes = kTile * 64 * 2;  // 64 dims of a tile: one swizzled block
  static constexpr int slots = D == 128 ? (NT == 2 ? 5 : 3) : (NT == 2 ? 8 : 6);  // K/V ring
  static constexpr size_t smem = 1024 + (NT + slots) * (size_t)tile_bytes + 512;
};

struct AttnTcArgs {
  // packed prompts
  const int32_t *cu_q, *cu_k;
  int n_seq, n_q, n_k;
  uint16_t* out;
  int64_t o_token, o_head;
  float* lse;
  const uint16_t *q, *k, *v;  // as the tensor maps have them (see kept_apart)
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  // shared prefix
  const int32_t* pages;
  int n_prefix_pages, n_pages, shift, prefix_len, n_rows, splits, tiles_per_split;
  float* part_o;
  float2* part_ml;
  // both
  int Hq, Hkv, grp, tpt;  // query heads per KV head; tokens (rows) per row tile
  float c;                // scale * log2 e
  int* err;               // where a wait that gives up says so; null: this file's word
};

__device__ __forceinline__ uint64_t kdesc(uint32_t addr) {
  // K-major, 128-byte swizzle: 8-row groups 1024 bytes apart
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t vdesc(uint32_t addr, uint32_t block) {
  // MN-major (V: the contiguous dims are the product's columns), 128-byte
  // swizzle: 64-dim blocks `block` bytes apart, 8-key groups 1024 bytes apart
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(block >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
template <int F16, int N, int BMN>
constexpr uint32_t tc_idesc() {
  return (1u << 4) | ((uint32_t)!F16 << 7) | ((uint32_t)!F16 << 10) | ((uint32_t)BMN << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// One lane of a converged warp (the same one each time).  Unlike lane == 0 it
// lets the compiler keep descriptors in uniform registers: an MMA then issues
// in fewer cycles than it runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define M3_R32(r)                                                                               \
  r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], r[12], r[13], r[14], \
      r[15], r[16], r[17], r[18], r[19], r[20], r[21], r[22], r[23], r[24], r[25], r[26], r[27], \
      r[28], r[29], r[30], r[31]

// 32 columns of this thread's lane.  The values may be used after ld_wait and
// then ld_touch, which ties them to a point behind the wait.
__device__ __forceinline__ void tm_ld(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void ld_touch(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                 "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tm_st(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* tm, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* tm, int x, int y, int z, int w,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// What a CTA works on.
struct TcWork {
  int h;          // KV head
  int first[2];   // first token (row) of each row tile
  int count[2];   // its tokens
  int n[2];       // key tiles of each
  int key0;       // first key of key tile 0: a row of k and v, or a prefix position
  int hi;         // keys past key0 that exist for these rows
  int pos0;       // packed: the first tile's first token sits at key pos0
  int split;
  int fix;        // the key tile that reaches past them, or -1
};

// Packed: the CTA's NT x tpt tokens.  Sequences are walked 32 at a time.
template <int NT>
__device__ __forceinline__ bool find_prompt_work(const AttnTcArgs& a, int w, int lane, TcWork& k) {
  const int span = NT * a.tpt;
  int before = 0;
  for (int s0 = 0; s0 < a.n_seq; s0 += 32) {
    const int s = s0 + lane;
    int qa = 0, lq = 0, units = 0;
    if (s < a.n_seq) {
      qa = min(max(a.cu_q[s], 0), a.n_q);
      lq = max(min(a.cu_q[s + 1], a.n_q) - qa, 0);
      units = (lq + span - 1) / span;
    }
    int inc = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += v;
    }
    const int all = __shfl_sync(~0u, inc, 31);
    if (w < before + all) {
      const unsigned hit = __ballot_sync(~0u, w < before + inc);
      const int src = __ffs(hit) - 1;
      const int u = __shfl_sync(~0u, w - before - (inc - units), src);  // the unit in its sequence
      qa = __shfl_sync(~0u, qa, src);
      lq = __shfl_sync(~0u, lq, src);
      units = __shfl_sync(~0u, units, src);
      const int seq = s0 + src;
      int ka = qa, lk = lq;
      if (a.cu_k) {
        ka = min(max(a.cu_k[seq], 0), a.n_k);
        lk = max(min(a.cu_k[seq + 1], a.n_k) - ka, 0);
      } else {
        lk = max(min(qa + lq, a.n_k) - ka, 0);
      }
      const int t0 = (units - 1 - u) * span;  // the longest rows first
      k.pos0 = t0 + lk - lq;
      k.key0 = ka;
      k.hi = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        k.first[t] = qa + t0 + t * a.tpt;
        k.count[t] = t < NT ? min(max(lq - t0 - t * a.tpt, 0), a.tpt) : 0;
        const int keys = k.count[t] ? max(k.pos0 + t * a.tpt + k.count[t], 0) : 0;
        k.n[t] = (keys + kTile - 1) / kTile;
        k.hi = max(k.hi, keys);
      }
      return true;
    }
    before += all;
  }
  return false;
}

// Values of keys that a row does not attend to come to it through 0 * v in the
// key tile on the diagonal, which is not 0 for an infinity or a NaN.  For 32
// columns of o that hold one: if such a key is where it came from, the row is
// summed again over its own keys alone, with the same m, one by one.  Slow, and
// reached by such values only.
template <int D, int F16>
__device__ __forceinline__ void kept_apart(const AttnTcArgs& a, int h, int head, int at, int key0,
                                           int keys, int end, int col, float mc, uint32_t* o) {
  constexpr uint32_t kMask = F16 ? 0x7C00u : 0x7F80u;  // an exponent of ones: no number
  const uint16_t* v = a.v + (int64_t)key0 * a.v_token + (int64_t)h * a.v_head + col;
  bool strange = false;
  for (int j = max(keys, 0); j < end && !strange; ++j) {
    const uint4* x = reinterpret_cast<const uint4*>(v + (int64_t)j * a.v_token);
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      const uint4 y = __ldg(x + e);
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int b = 0; b < 4; ++b)
        strange |= (w[b] & kMask) == kMask || ((w[b] >> 16) & kMask) == kMask;
    }
  }
  if (!strange) return;
  const uint4* q = reinterpret_cast<const uint4*>(a.q + (int64_t)at * a.q_token +
                                                  (int64_t)head * a.q_head);
  const uint16_t* k = a.k + (int64_t)key0 * a.k_token + (int64_t)h * a.k_head;
  float y[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) y[e] = 0.0f;
#pragma unroll 1
  for (int j = 0; j < keys; ++j) {
    const uint4* kj = reinterpret_cast<const uint4*>(k + (int64_t)j * a.k_token);
    const uint4* vj = reinterpret_cast<const uint4*>(v + (int64_t)j * a.v_token);
    float s = 0.0f;
#pragma unroll 1
    for (int d = 0; d < D / 8; ++d) {
      const uint4 x = __ldg(q + d), z = __ldg(kj + d);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float2 u = unpack2<F16>(xs[b]), w = unpack2<F16>(zs[b]);
        s = fmaf(u.x, w.x, fmaf(u.y, w.y, s));
      }
    }
    const float p = unpack2<F16>(pack2<F16>(ex2(fmaf(s, a.c, -mc)), 0.0f)).x;
    bool nan = true;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint4 z = __ldg(vj + d);
      const uint32_t zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float2 w = unpack2<F16>(zs[b]);
        const int e = 8 * d + 2 * b;
        y[e] = fmaf(p, w.x, y[e]);
        y[e + 1] = fmaf(p, w.y, y[e + 1]);
        nan = nan && y[e] != y[e] && y[e + 1] != y[e + 1];
      }
    }
    if (nan) break;  // and so they stay
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(y[e]);
}

template <int D, int F16, bool PAGED, int NT>
__global__ void __launch_bounds__(384, 1)  // 168 registers, with one row tile (256 threads) too
    attn_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const AttnTcArgs a) {
  using S = TcShape<D, NT>;
  constexpr int NS = S::slots;
  extern __shared__ uint8_t tc_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)tc_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;                         // NT row tiles
  uint8_t* skv = smem + NT * S::tile_bytes;    // ring: K 0, V 0, K 1, V 1, ...
  uint64_t* full = reinterpret_cast<uint64_t*>(skv + NS * (size_t)S::tile_bytes);
  uint64_t* empty = full + NS;
  uint64_t* qfull = empty + NS;
  uint64_t* sfull = qfull + 1;   // [2] S of a row tile is there
  uint64_t* pfull = sfull + 2;   // [2][2] P is written: keys 0..63, 64..127
  uint64_t* ofull = pfull + 4;   // [2] the last product is done
  uint64_t* vfix = ofull + 2;    // the rows past the last key are cleared
  uint64_t* drain = vfix + 1;    // [2]
  uint64_t* turn = drain + 2;    // [2] whose products are next
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(turn + 2);
  int* counts = reinterpret_cast<int*>(tmem_slot + 1);  // tiles asked for, seen by each MMA warp
  uint32_t* seen_mask = reinterpret_cast<uint32_t*>(counts + 3);  // [8] 16-key pieces of a key tile
  __shared__ TcWork work;
  __shared__ int have_work;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* err = a.err ? a.err : &g_ops_err;
  if (warp == 0) {
    TcWork k;
    bool some;
    if constexpr (PAGED) {
      k.split = blockIdx.x % a.splits;
      const int r = blockIdx.x / a.splits;
      k.h = r % a.Hkv;
      const int unit = r / a.Hkv;
      const int all = (a.prefix_len + kTile - 1) / kTile;
      const int j0 = min(all, k.split * a.tiles_per_split);
      const int nj = min(all - j0, a.tiles_per_split);
      k.key0 = j0 * kTile;
      k.hi = a.prefix_len - k.key0;
      k.pos0 = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        k.first[t] = (unit * NT + t) * a.tpt;
        k.count[t] = t < NT ? min(max(a.n_rows - k.first[t], 0), a.tpt) : 0;
        k.n[t] = k.count[t] ? nj : 0;
      }
      some = true;
    } else {
      some = find_prompt_work<NT>(a, blockIdx.x / a.Hkv, lane, k);
      k.h = blockIdx.x % a.Hkv;
      k.split = 0;
    }
    if (lane == 0) {
      have_work = some;
      if (some) {
        const int n = max(k.n[0], k.n[1]);
        k.fix = k.hi < n * kTile ? n - 1 : -1;
        work = k;
      }
      for (int s = 0; s < NS; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], NT);
      }
      mbar_init(qfull, 1);
      mbar_init(vfix, 1);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&sfull[t], 1);
        mbar_init(&drain[t], 1);
        mbar_init(&turn[t], 1);
        mbar_init(&pfull[2 * t], 4);
        mbar_init(&pfull[2 * t + 1], 4);
        mbar_init(&ofull[t], 1);
      }
      counts[0] = counts[1] = counts[2] = 0;
      fence_barrier_init();
    }
  }
  __syncthreads();
  // (m3_attn_prefix: the row's own positions need nothing from here)
  if constexpr (PAGED) pdl_launch_dependents();
  if (!have_work) return;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(S::columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const TcWork& w = work;  // in shared memory: indexed by the row tile
  const int n_max = max(w.n[0], w.n[1]);
  // columns: S (and P over it) of row tile t at 128 t, O at 128 (NT + t)
  const uint32_t idesc_s = tc_idesc<F16, kTile, 0>(), idesc_o = tc_idesc<F16, D, 1>();

  // the softmax holds a row of S in registers: it takes them from the other
  // four warps (NT = 2: 128 x 72 + 256 x 216 = 384 x 168, the launch's own
  // total; NT = 1: 128 x 72 + 128 x 216 < 256 x 168)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ------------------------------------------------------------- TMA --
    if (warp == 0 && n_max > 0) {
      if (lane == 0) {
        const uint32_t qbytes = (uint32_t)(a.grp * a.tpt) * D * 2;
        mbar_arrive_expect_tx(qfull, ((w.n[0] > 0) + (w.n[1] > 0)) * qbytes);
        for (int t = 0; t < NT; ++t)
          if (w.n[t] > 0)
            for (int c = 0; c < D / 64; ++c)
              tma_3d(sq + t * S::tile_bytes + c * S::half_bytes, &tq, c * 64, w.h * a.grp,
                     w.first[t], qfull);
      }
      // paged: lane i brings the i-th page (or its 128 places) of a key tile;
      // its number is asked for one tile ahead
      const int page = 1 << a.shift, box = min(page, kTile), boxes = kTile / box;
      auto number_of = [&](int j) -> int {
        const long long at = (long long)w.key0 + (long long)j * kTile + lane * box;
        if (lane >= boxes || at >= a.prefix_len || (at >> a.shift) >= a.n_prefix_pages) return -1;
        const int x = __ldg(a.pages + (at >> a.shift));
        return x >= a.n_pages ? -1 : x;
      };
      int number = PAGED ? number_of(0) : 0;
      bool ok = true;
      int it = 0, slot = 0;
      uint32_t phase = 1;  // the first round finds every slot empty
      for (int j = 0; j < n_max && ok; ++j) {
        int x = 0, off = 0;
        if constexpr (PAGED) {
          // a page that is not there: past the pool, which reads as zeros, and
          // left out of the softmax
          const unsigned there = __ballot_sync(~0u, number >= 0);
          if (lane == 0) {
            uint32_t m = 0;
            for (int i = 0; i < boxes; ++i)
              if ((there >> i) & 1) m |= ((1u << (box / 16)) - 1) << (i * (box / 16));
            seen_mask[j & 7] = m;
          }
          x = number < 0 ? a.n_pages : number;
          off = (w.key0 + j * kTile + lane * box) & (page - 1);
          number = number_of(j + 1);
        }
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && mbar_wait(&empty[slot], phase, err);
          if (!ok) break;
          uint8_t* dst = skv + (size_t)slot * S::tile_bytes;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], S::tile_bytes);
          __syncwarp();
          if constexpr (PAGED) {
            if (lane < boxes)
              for (int c = 0; c < D / 64; ++c)
                tma_4d(dst + c * S::half_bytes + lane * box * 128, &tk, c * 64, off,
                       w.h + kv * a.Hkv, x, &full[slot]);
          } else if (lane < D / 64) {
            tma_3d(dst + lane * S::half_bytes, kv ? &tv : &tk, lane * 64, w.h,
                   w.key0 + j * kTile, &full[slot]);
          }
          ++it;
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (lane == 0) counts[0] = it;
    }
    if (warp == 0 && w.fix >= 0) {
      // what lies past the keys in the last tile may be anything, and 0 * NaN
      // is not 0: those rows of V are cleared.  (By this warp, which has seen
      // the slot's earlier uses end: another could take an earlier phase of
      // the barrier for this one.)
      __syncwarp();
      const int i = 2 * w.fix + 1, rows = w.hi - w.fix * kTile;
      if (mbar_wait(&full[i % NS], (uint32_t)(i / NS) & 1u, err)) {
        uint8_t* v = skv + (size_t)(i % NS) * S::tile_bytes;
        for (int p = rows * 8 + lane; p < kTile * 8; p += 32)
          for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<uint4*>(v + c * S::half_bytes + p * 16) = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(vfix);
    }
    // ------------------------------------------------------------- MMA --
    // A warp per row tile: the waits of one tile hide behind the products of
    // the other.  Both see every K/V tile, since both have to give it back.
    // They take turns, O += P V and the next S = Q K^T of one tile together:
    // left alone the tiles fall into step, and then both softmaxes compete for
    // the exponentials while the tensor cores wait.
    if (warp >= 1 && warp <= NT && n_max > 0) {
      const int t = warp - 1, mine = w.n[t];
      const uint32_t ts = tmem + t * kTile, to = tmem + (NT + t) * kTile;
      const uint64_t dq = kdesc(smem_u32(sq + t * S::tile_bytes)), dk = kdesc(smem_u32(skv));
      const uint64_t dv = vdesc(smem_u32(skv), S::half_bytes);
      int slot = 0, seen = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto wait_tile = [&]() {  // the next tile of the ring
        ok = ok && mbar_wait(&full[slot], phase, err);
        seen += ok;
      };
      auto give_back = [&]() {  // once this thread's MMAs so far are done
        mma_commit(&empty[slot]);
      };
      auto next_slot = [&]() {
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      };
      auto scores = [&]() {  // S = Q K^T
        const uint64_t b0 = dk + (uint64_t)slot * (S::tile_bytes >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks / 4) * S::half_bytes + (ks % 4) * 32) >> 4;
          mma_ss(ts, dq + off, b0 + off, idesc_s, ks > 0);
        }
        mma_commit(&sfull[t]);
      };
      ok = mbar_wait(qfull, 0, err);
      wait_tile();
      fence_after();
      if (ok && elect_one()) {
        if (mine > 0) scores();
        give_back();
      }
      __syncwarp();
      next_slot();
      for (int j = 0; j < n_max && ok; ++j) {
        wait_tile();
        if (ok && j == w.fix) ok = mbar_wait(vfix, 0, err);
        const uint64_t b0 = dv + (uint64_t)slot * (S::tile_bytes >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (j < mine) ok = ok && mbar_wait(&pfull[2 * t + half], (uint32_t)j & 1u, err);
          // (a warp without work waits too: it must not run two turns ahead)
          if (NT == 2 && !half && (t || j))
            ok = ok && mbar_wait(&turn[t], (uint32_t)(j + t + 1) & 1u, err);
          if (j >= mine) break;
          fence_after();
          if (ok && elect_one()) {
#pragma unroll
            for (int k4 = 0; k4 < kTile / 32; ++k4) {  // 16 keys a step: 2048 bytes of V rows
              const int ks = half * (kTile / 32) + k4;
              mma_ts(to, ts + ks * 8, b0 + ks * (2048 >> 4), idesc_o, (j > 0 || ks > 0));
            }
            if (half) {
              give_back();
              if (j + 1 == mine) mma_commit(&ofull[t]);
            }
          }
          __syncwarp();
        }
        if (ok && j >= mine && elect_one()) give_back();
        __syncwarp();
        next_slot();
        if (!ok) break;
        if (j + 1 < n_max) {
          wait_tile();
          fence_after();
          if (ok && elect_one()) {
            if (j + 1 < mine) scores();
            give_back();
          }
          __syncwarp();
          next_slot();
        }
        if (NT == 2 && lane == 0) mbar_arrive(&turn[1 - t]);
      }
      if (!ok && elect_one()) {  // this thread's MMAs finish before the memory goes away
        mma_commit(&drain[t]);
        for (long long i = 0; i < kSpinLimit && !mbar_try_wait(&drain[t], 0); ++i) {
        }
      }
      if (lane == 0) counts[1 + t] = seen;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // --------------------------------------------------------- softmax --
    const int t = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t base = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t ts = base + t * kTile, to = base + (NT + t) * kTile;
    const int tok = row / a.grp, head = w.h * a.grp + row % a.grp, tiles = w.n[t];
    const bool mine = tok < w.count[t] && row < a.grp * a.tpt;
    // keys this row attends to, counted from key0
    const int keys = PAGED ? w.hi : w.pos0 + t * a.tpt + tok + 1;
    float m = -INFINITY, l = 0.0f;  // reference maximum (of q.k), sum of 2^((s - m) c)
    bool ok = true;
    for (int j = 0; j < tiles; ++j) {
      ok = mbar_wait(&sfull[t], (uint32_t)j & 1u, err);
      if (!ok) break;
      fence_after();
      uint32_t s[kTile];
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      const int lim = keys - j * kTile;
      uint32_t there = 0xFFu;
      if constexpr (PAGED) there = *reinterpret_cast<volatile uint32_t*>(&seen_mask[j & 7]);
      const bool cut = lim < kTile || there != 0xFFu;
#pragma unroll
      for (int k = 0; k < 4; ++k) tm_ld(ts + 32 * k, s + 32 * k);
      ld_wait();
#pragma unroll
      for (int k = 0; k < 4; ++k) ld_touch(s + 32 * k);
      if (cut) {
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          s[i] = i < lim && ((there >> (i / 16)) & 1) ? s[i] : 0xFF800000u;
      }
#pragma unroll
      for (int i = 0; i < kTile; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mx[e] = max3(mx[e], __uint_as_float(s[i + 2 * e]), __uint_as_float(s[i + 2 * e + 1]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool raise = (top - m) * a.c > kRaise || (m == -INFINITY && top > m);
      if (__any_sync(~0u, raise)) {
        const float f = raise ? ex2((m - top) * a.c) : 1.0f;  // 0 where m = -inf
        if (raise) m = top;
        l *= f;
        if (j > 0) {
          // S of this tile is complete, so the products before it are: O is ours
#pragma unroll
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tm_ld(to + i, o);
            ld_wait();
            ld_touch(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tm_st(to + i, o);
          }
        }
      }
      const float mc = m == -INFINITY ? 0.0f : m * a.c;
      const uint64_t c2 = pack_f32x2(a.c, a.c), mc2 = pack_f32x2(-mc, -mc);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < kTile; i += 64) {
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 z = unpack_f32x2(fma2(pack_u32x2(s[i + 2 * e], s[i + 2 * e + 1]), c2, mc2));
          const float x = ex2(z.x), y = ex2(z.y);
          fadd2(sum[e & 1], pack_f32x2(x, y));
          p[e] = pack2<F16>(x, y);  // the weights in the operand type of the product with V
        }
        tm_st(ts + i / 2, p);
        // half of the keys: their product may start
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * t + i / 64]);
      }
      fadd2(sum[0], sum[1]);
      const float2 sums = unpack_f32x2(sum[0]);
      l += sums.x + sums.y;
    }
    // ----------------------------------------------------------- output --
    if (tiles > 0 && ok) {
      ok = mbar_wait(&ofull[t], 0, err);
      fence_after();
    }
    if (ok) {
      const bool some = tiles > 0;
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      if constexpr (PAGED) {
        const size_t id = (size_t)w.split * a.n_rows * a.Hq + (size_t)(w.first[t] + tok) * a.Hq + head;
        if (mine) a.part_ml[id] = make_float2(m * a.c, l);
#pragma unroll
        for (int i = 0; i < D; i += 32) {
          if (!some) break;
          uint32_t o[32];
          tm_ld(to + i, o);
          ld_wait();
          ld_touch(o);
          if (mine) {
            uint4* p = reinterpret_cast<uint4*>(a.part_o + id * D + i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              p[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      } else {
        const size_t at = (size_t)w.first[t] + tok;
        if (mine && a.lse)
          a.lse[at * a.Hq + head] = l == 0.0f ? -INFINITY : (m * a.c + log2f(l)) * kLn2;
        uint16_t* dst = a.out + (int64_t)at * a.o_token + (int64_t)head * a.o_head;
        float zero = 0.0f;  // or NaN, where o holds an infinity or a NaN
        auto store = [&](int i, const uint32_t* o) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[e] = some && inv != 0.0f ? pack2<F16>(__uint_as_float(o[2 * e]) * inv,
                                                    __uint_as_float(o[2 * e + 1]) * inv)
                                       : 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(dst + i + 8 * e) =
                make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        };
#pragma unroll
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          if (some) {
            tm_ld(to + i, o);
            ld_wait();
            ld_touch(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) zero = fmaf(__uint_as_float(o[e]), 0.0f, zero);
          }
          if (mine) store(i, o);
        }
        const bool strange = mine && zero != 0.0f && l > 0.0f;
        if (__any_sync(~0u, strange)) {
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tm_ld(to + i, o);
            ld_wait();
            ld_touch(o);
            if (strange) {
              kept_apart<D, F16>(a, w.h, head, (int)at, w.key0, keys, min(w.hi, tiles * kTile), i,
                                 m == -INFINITY ? 0.0f : m * a.c, o);
              store(i, o);
            }
          }
        }
      }
    }
    fence_before();
  }

  __syncthreads();
  if (tid == 0 && n_max > 0) {
    // copies asked for but never seen (only after a failed wait): let them land
    for (long long k = 0; k < kSpinLimit && !mbar_try_wait(qfull, 0); ++k) {
    }
    for (int i = NT == 2 ? min(counts[1], counts[2]) : counts[1]; i < counts[0]; ++i)
      for (long long k = 0; k < kSpinLimit && !mbar_try_wait(&full[i % NS], (uint32_t)(i / NS) & 1u);
           ++k) {
      }
  }
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(S::columns)
                 : "memory");
  }
}

// --------------------------------------------------- a row's own positions --
// One CTA: the (up to 16) query heads of one KV head of one row against a run
// of its positions, or of the prefix's where that is short.  Each of 4 warps takes every 4th 16-position tile, K and
// V by 16-byte asynchronous copies into its own ring, swizzled for ldmatrix;
// S = Q K^T and O += P V on m16n8k16, fp32 softmax.  Positions past the length
// and pages that are not there are filled with zeros, not read, and masked.
// Bound by HBM: 16 rows of 700 to 4500 positions, 8 KV heads of 128, alone 136 MB
// in 27 us, 5.0 TB/s, with the ramp at both ends; more, smaller CTAs measured
// slower (8 per SM 40.7 against 37.4 us for the whole call).
constexpr int kOwnWarps = 4;
constexpr int kOwnTile = 16;
constexpr int kOwnStages = 3;
constexpr int kClusterMost = 8;  // splits that a cluster joins

template <int D>
constexpr size_t own_smem() {
  const size_t ring = (size_t)kOwnWarps * kOwnStages * 2 * kOwnTile * D * 2;
  const size_t merge = (size_t)(kOwnWarps + 1) * 16 * (D + 2) * 4;
  return ring > merge ? ring : merge;
}

struct OwnArgs {
  const uint16_t* q;
  int64_t q_row, q_head;
  const uint16_t* pool;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int n_pages, shift, max_pages;
  const int32_t* prefix_pages;  // pre_splits > 0: the prefix, read by every row for itself
  int prefix_len, pre_splits;
  int n_rows, Hq, Hkv, grp, mtiles, splits;  // splits: of the prefix, then of the own positions
  float c;
  float* part_o;    // [splits][n_rows * Hq][D]
  float2* part_ml;  // [splits][n_rows * Hq]
  // the splits of a row in one cluster: its result
  uint16_t* out;
  int64_t o_row, o_head;
  float* lse;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

// CLUSTER: the splits of a row and KV head are a cluster, which joins them
// through its shared memory and writes the row itself.
template <int D, int F16, bool CLUSTER>
__global__ void __launch_bounds__(kOwnWarps * 32) attn_own_kernel(const OwnArgs a) {
  constexpr int ROWB = D * 2, KS = D / 16, NTO = D / 8, CH = D / 8;
  extern __shared__ __align__(128) uint8_t own_raw[];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  int x = blockIdx.x;
  const int split = x % a.splits;
  x /= a.splits;
  const int mt = x % a.mtiles;
  x /= a.mtiles;
  const int g = x % a.Hkv, b = x / a.Hkv;
  const bool pre = split < a.pre_splits;
  const int len = pre ? a.prefix_len
                      : (int)min((long long)max(a.lens[b], 0), (long long)a.max_pages << a.shift);
  const int tiles = (len + kOwnTile - 1) / kOwnTile;
  const int of = pre ? a.pre_splits : a.splits - a.pre_splits;
  const int per = (tiles + of - 1) / of;
  const int t0 = min(tiles, (pre ? split : split - a.pre_splits) * per);
  const int t1 = min(tiles, t0 + per);
  const size_t rows = (size_t)a.n_rows * a.Hq;
  const int heads = min(16, a.grp - mt * 16);
  const size_t id0 = (size_t)split * rows + (size_t)b * a.Hq + g * a.grp + mt * 16;
  if (!CLUSTER && t0 >= t1) {
    if (tid < heads) a.part_ml[id0 + tid] = make_float2(-INFINITY, 0.0f);
    if (blockIdx.x == 0) pdl_wait();
    return;
  }
  uint8_t* ring = own_raw + (size_t)warp * kOwnStages * 2 * kOwnTile * ROWB;
  const uint32_t ring_u = smem_u32(ring);
  const int nmine = t1 - t0 > warp ? (t1 - t0 - warp + kOwnWarps - 1) / kOwnWarps : 0;
  const int32_t* trow = pre ? a.prefix_pages : a.table + (size_t)b * a.ld_table;
  const size_t page_elems = (size_t)2 * a.Hkv * D << a.shift;
  // the page numbers of this warp's tiles, 32 tiles at a time (one per lane)
  int held = -1;
  auto page_of = [&](int i) -> int {
    if ((i & 31) == 0) {
      const int t = t0 + warp + (i + lane) * kOwnWarps;
      held = t < t1 ? trow[(t * kOwnTile) >> a.shift] : -1;
      if (held >= a.n_pages) held = -1;
    }
    return __shfl_sync(~0u, held, i & 31);
  };
  uint32_t live = 0;  // bit (i % 32): tile i has its page
  // a lane's 16-byte pieces: row lr + RPP e, piece lc, e < PPL; the swizzle
  // piece ^ (row & 7) takes its lane and its e apart
  constexpr int RPP = 32 / CH, PPL = kOwnTile / RPP;
  const int lr = lane / CH, lc = lane % CH;
  const uint32_t lane_src = lr * D + lc * 8, lane_dst = lr * ROWB;
  const uint32_t lane_piece = lc ^ (lr & 7);
  auto fetch = [&](int i) {
    if (i < nmine) {
      const int t = t0 + warp + i * kOwnWarps;
      const int page = page_of(i);
      live = page >= 0 ? live | (1u << (i & 31)) : live & ~(1u << (i & 31));
      const int p0 = t * kOwnTile, off = p0 & ((1 << a.shift) - 1);
      const uint16_t* kp = a.pool + (size_t)max(page, 0) * page_elems +
                           (((size_t)g << a.shift) + off) * D + lane_src;
      const uint16_t* vp = kp + ((size_t)a.Hkv << a.shift) * D;
      const uint32_t dst = ring_u + (i % kOwnStages) * 2 * kOwnTile * ROWB + lane_dst;
      const int nv = page >= 0 ? len - p0 : 0;  // rows of the tile that are there
      if (nv >= kOwnTile) {
#pragma unroll
        for (int e = 0; e < PPL; ++e) {
          const uint32_t o = e * RPP * ROWB + ((lane_piece ^ ((e * RPP) & 7)) << 4);
          cp16(dst + o, kp + e * RPP * D, true);
          cp16(dst + kOwnTile * ROWB + o, vp + e * RPP * D, true);
        }
      } else {  // zeros past them, and nothing read
#pragma unroll
        for (int e = 0; e < PPL; ++e) {
          const uint32_t o = e * RPP * ROWB + ((lane_piece ^ ((e * RPP) & 7)) << 4);
          const bool there = lr + e * RPP < nv;
          const int back = there ? e * RPP * D : -(int)lane_src;
          cp16(dst + o, kp + back, there);
          cp16(dst + kOwnTile * ROWB + o, vp + back, there);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kOwnStages - 1; ++i) fetch(i);

  // Q fragments: rows gid and gid + 8 are heads of the group
  uint32_t qa[KS][4];
  {
    const uint16_t* q0 = a.q + (int64_t)b * a.q_row + (int64_t)(g * a.grp + mt * 16) * a.q_head;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = gid + 8 * (e & 1), d = ks * 16 + 2 * tig + 8 * (e >> 1);
        qa[ks][e] = r < heads ? *reinterpret_cast<const uint32_t*>(q0 + r * a.q_head + d) : 0u;
      }
  }
  float o[NTO][4];
#pragma unroll
  for (int j = 0; j < NTO; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // m in log2 units

  for (int i = 0; i < nmine; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kOwnStages - 2) : "memory");
    __syncwarp();
    const bool there = (live >> (i & 31)) & 1;
    fetch(i + kOwnStages - 1);  // into the slot that tile i - 1 has left
    if (!there) continue;
    const uint32_t kb = ring_u + (i % kOwnStages) * 2 * kOwnTile * ROWB;
    const uint32_t vb = kb + kOwnTile * ROWB;
    const int nv = min(kOwnTile, len - (t0 + warp + i * kOwnWarps) * kOwnTile);
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
      const int prow = 8 * j + (lane & 7);
#pragma unroll
      for (int kk = 0; kk < KS; kk += 2) {
        const int ch = 2 * kk + (lane >> 3);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kb + prow * ROWB + ((ch ^ (prow & 7)) << 4), b0, b1, b2, b3);
        mma16816<F16>(s[j], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
        mma16816<F16>(s[j], qa[kk + 1][0], qa[kk + 1][1], qa[kk + 1][2], qa[kk + 1][3], b2, b3);
      }
    }
    if (nv < kOwnTile) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * j + 2 * tig + (e & 1) >= nv) s[j][e] = -INFINITY;
    }
    // the reference maximum is raised only past 2^kRaise, as in attn_tc_kernel
    float f[2] = {1.0f, 1.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1])) * a.c;
      x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
      x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
      if (x - m[h] > kRaise || (m[h] == -INFINITY && x > m[h])) {
        f[h] = ex2(m[h] - x);
        m[h] = x;
      }
    }
    const float r0 = m[0] == -INFINITY ? 0.0f : m[0], r1 = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = ex2(fmaf(s[j][e], a.c, (e >> 1) ? -r1 : -r0));
    // this lane's share of the rows' sums
    l[0] = l[0] * f[0] + ((s[0][0] + s[0][1]) + (s[1][0] + s[1][1]));
    l[1] = l[1] * f[1] + ((s[0][2] + s[0][3]) + (s[1][2] + s[1][3]));
    if (__any_sync(~0u, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
      for (int j = 0; j < NTO; ++j) {
        o[j][0] *= f[0];
        o[j][1] *= f[0];
        o[j][2] *= f[1];
        o[j][3] *= f[1];
      }
    }
    const uint32_t p0 = pack2<F16>(s[0][0], s[0][1]), p1 = pack2<F16>(s[0][2], s[0][3]);
    const uint32_t p2 = pack2<F16>(s[1][0], s[1][1]), p3 = pack2<F16>(s[1][2], s[1][3]);
    const int prow = (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
    for (int j = 0; j < NTO; j += 2) {
      const int ch = j + (lane >> 4);
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(vb + prow * ROWB + ((ch ^ (prow & 7)) << 4), b0, b1, b2, b3);
      mma16816<F16>(o[j], p0, p1, p2, p3, b0, b1);
      mma16816<F16>(o[j + 1], p0, p1, p2, p3, b2, b3);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(~0u, l[h], 1);
    l[h] += __shfl_xor_sync(~0u, l[h], 2);
  }
  // the warps' results meet in shared memory (the rings are done with)
  __syncthreads();
  float* mo = reinterpret_cast<float*>(own_raw);        // [warp][16][D]
  float* mml = mo + kOwnWarps * 16 * D;                 // [warp][16][2]
  float* co = mml + kOwnWarps * 16 * 2;                 // CLUSTER: the CTA's own [16][D]
  float* cml = co + 16 * D;                             // [16][2]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = gid + 8 * h;
    if (r < heads) {
      float* dst = mo + (warp * 16 + r) * D;
#pragma unroll
      for (int j = 0; j < NTO; ++j)
        *reinterpret_cast<float2*>(dst + j * 8 + 2 * tig) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
      if (tig == 0) {
        mml[(warp * 16 + r) * 2] = m[h];
        mml[(warp * 16 + r) * 2 + 1] = l[h];
      }
    }
  }
  __syncthreads();
  for (int r = warp; r < heads; r += kOwnWarps) {
    // A warp without a key has the sum 0, marked by a factor below 0.  Scores
    // that are NaN leave the maximum as it is and make the sum NaN, whatever its
    // factor.
    float mm = -INFINITY, f[kOwnWarps], ll = 0.0f;
#pragma unroll
    for (int k = 0; k < kOwnWarps; ++k) mm = fmaxf(mm, mml[(k * 16 + r) * 2]);
#pragma unroll
    for (int k = 0; k < kOwnWarps; ++k) {
      const float mk = mml[(k * 16 + r) * 2], lk = mml[(k * 16 + r) * 2 + 1];
      f[k] = lk == 0.0f ? -1.0f : ex2(mk - mm);
      if (lk != 0.0f) ll += lk * f[k];
    }
    for (int d = lane; d < D; d += 32) {
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < kOwnWarps; ++k)
        if (f[k] >= 0.0f) y += mo[(k * 16 + r) * D + d] * f[k];
      if constexpr (CLUSTER) co[r * D + d] = y;
      else a.part_o[(id0 + r) * D + d] = y;
    }
    if (lane == 0) {
      if constexpr (CLUSTER) {
        cml[2 * r] = mm;
        cml[2 * r + 1] = ll;
      } else {
        a.part_ml[id0 + r] = make_float2(mm, ll);
      }
    }
  }
  if constexpr (CLUSTER) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    // head by head over the cluster's CTAs, a warp each
    const bool padding = a.lens[b] < 0;
    for (int r = split * kOwnWarps + warp; r < heads && !padding; r += a.splits * kOwnWarps) {
      // lane k has the max and sum of CTA k; a CTA without a key has (-inf, 0), o = 0
      float mk = -INFINITY, ll = 0.0f, v[kClusterMost][D / 32];
      if (lane < a.splits) {
        const float2 ml = *reinterpret_cast<const float2*>(cluster.map_shared_rank(cml, lane) + 2 * r);
        mk = ml.x;
        ll = ml.y;
      }
#pragma unroll
      for (int k = 0; k < kClusterMost; ++k) {  // all on their way at once
        const float* o = cluster.map_shared_rank(co, min(k, a.splits - 1)) + r * D + 2 * lane;
#pragma unroll
        for (int i = 0; i < D / 32; i += 2) {
          const float2 x = *reinterpret_cast<const float2*>(o + 32 * i);
          v[k][i] = x.x;
          v[k][i + 1] = x.y;
        }
      }
      float mm = mk;
#pragma unroll
      for (int o = 4; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
      // (a factor may be 0 beside a far larger maximum, and takes the sum with it)
      const float f = ll == 0.0f ? 0.0f : ex2(mk - mm);
      const unsigned have = __ballot_sync(~0u, ll != 0.0f);  // with a key; not the lanes past the last
      ll *= f;
#pragma unroll
      for (int o = 4; o; o >>= 1) ll += __shfl_xor_sync(~0u, ll, o);
      mm = __shfl_sync(~0u, mm, 0);
      ll = __shfl_sync(~0u, ll, 0);
      float y[D / 32] = {};
#pragma unroll
      for (int k = 0; k < kClusterMost; ++k) {
        const float fk = __shfl_sync(~0u, f, k);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          if ((have >> k) & 1) y[i] += v[k][i] * fk;
      }
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
      const int head = g * a.grp + mt * 16 + r;
      uint16_t* dst = a.out + (int64_t)b * a.o_row + (int64_t)head * a.o_head;
#pragma unroll
      for (int i = 0; i < D / 32; i += 2)
        *reinterpret_cast<uint32_t*>(dst + 2 * lane + 32 * i) =
            ll == 0.0f ? 0u : pack2<F16>(y[i] * inv, y[i + 1] * inv);
      if (lane == 0 && a.lse)
        a.lse[(size_t)b * a.Hq + head] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
    cluster.sync();  // the others may still read this CTA's memory
    return;
  }
  // The launch before this one is the prefix, beside which this one ran.  One
  // CTA waits for its end, so that the end of this launch is that of both.
  if (blockIdx.x == 0) pdl_wait();
}

// ------------------------------------------------------------------ join ---
// A row and query head: the parts' (max, sum, unnormalised o), D / 4 lanes a
// part, the parts side by side, then one sum over those.  A few dependent reads
// of L2: 5 to 7 us at the end of a call, its launch hidden by the one before.
struct JoinArgs {
  const float* part_o;
  const float2* part_ml;
  const int32_t* lens;
  uint16_t* out;
  int64_t o_row, o_head;
  float* lse;
  int n_rows, Hq, parts;
};

constexpr int kJoinThreads = 128;
constexpr int kMaxParts = 256;

// WARPS per (row, query head): 4, or 1 where there are rows enough.
template <int D, int F16, int WARPS>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const JoinArgs a) {
  constexpr int T = 32 * WARPS, ROWS = kJoinThreads / T;  // threads per row, rows per CTA
  constexpr int W = D / 4, SIDE = T / W;                  // lanes per part, parts side by side
  __shared__ float f[ROWS][kMaxParts];
  __shared__ float red[2][kJoinThreads / 32];
  __shared__ float4 acc[ROWS][SIDE][W];
  const int tid = threadIdx.x % T, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = threadIdx.x / T;
  auto sync = [&]() {
    if constexpr (WARPS == 1) __syncwarp();
    else __syncthreads();
  };
  const size_t rows = (size_t)a.n_rows * a.Hq, id = (size_t)blockIdx.x * ROWS + r;
  pdl_wait();
  if (id >= rows) return;
  const int b = (int)(id / a.Hq), h = (int)(id % a.Hq);
  if (a.lens[b] < 0) return;  // padding
  float m = -INFINITY;
  for (int p = tid; p < a.parts; p += T) m = fmaxf(m, __ldcg(a.part_ml + p * rows + id).x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  if constexpr (WARPS > 1) {
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WARPS; ++k) m = fmaxf(m, red[0][k]);
  }
  float l = 0.0f;
  for (int p = tid; p < a.parts; p += T) {
    const float2 ml = __ldcg(a.part_ml + p * rows + id);
    // A part without a key has the sum 0 and no o: marked by a factor below 0.
    // Every other one counts, also with the factor 0: its sum or o may be NaN
    // (scores that are NaN leave the maximum as it is).
    const float x = ex2(ml.x - m);
    f[r][p] = ml.y == 0.0f ? -1.0f : x;
    if (ml.y != 0.0f) l += ml.y * x;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
  if (WARPS > 1 && lane == 0) red[1][warp] = l;
  sync();
  if constexpr (WARPS > 1) {
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) l += red[1][k];
  }
  const int side = tid / W, d = (tid % W) * 4;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int p = side; p < a.parts; p += SIDE) {
    const float x = f[r][p];
    if (x < 0.0f) continue;
    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (p * rows + id) * D + d));
    y.x += v.x * x;
    y.y += v.y * x;
    y.z += v.z * x;
    y.w += v.w * x;
  }
  if constexpr (SIDE > 1) {
    acc[r][side][tid % W] = y;
    sync();
  }
  if (tid < W) {
#pragma unroll
    for (int k = 1; k < SIDE; ++k) {
      const float4 v = acc[r][k][tid];
      y.x += v.x;
      y.y += v.y;
      y.z += v.z;
      y.w += v.w;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 o = make_uint2(0u, 0u);
    if (l != 0.0f) o = make_uint2(pack2<F16>(y.x * inv, y.y * inv), pack2<F16>(y.z * inv, y.w * inv));
    *reinterpret_cast<uint2*>(a.out + (int64_t)b * a.o_row + (int64_t)h * a.o_head + d) = o;
    if (tid == 0 && a.lse) a.lse[id] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// ------------------------------------------------------------------ host ---
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Boxes of 64 dims x box[1] x box[2] (x box[3]) in the 128-byte swizzle.
bool make_map(CUtensorMap* tm, int f16, int rank, const void* base, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
  auto fn = encode_fn();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn && fn(tm, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [n][heads][D] with strides (elements), boxes of `rows` x `heads_box` x 64.
bool make_rows_map(CUtensorMap* tm, int f16, const void* base, int n, int heads, int D,
                   int64_t s_row, int64_t s_head, int heads_box, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)n};
  const cuuint64_t strides[2] = {(cuuint64_t)s_head * 2, (cuuint64_t)s_row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows};
  return make_map(tm, f16, 3, base, dims, strides, box);
}

// A kernel's shared-memory limit, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  // all of the SM's memory as shared memory, or two kernels' CTAs could not
  // stand side by side on it
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

template <int D, int F16, bool PAGED, int NT>
cudaError_t launch_tc_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const AttnTcArgs& a, unsigned grid, cudaStream_t st) {
  using S = TcShape<D, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(attn_tc_kernel<D, F16, PAGED, NT>, S::smem, done);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<D, F16, PAGED, NT><<<grid, S::threads, S::smem, st>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

template <bool PAGED, int NT>
cudaError_t launch_tc_n(int D, int f16, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const AttnTcArgs& a, unsigned grid, cudaStream_t st) {
  if (D == 128)
    return f16 ? launch_tc_t<128, 1, PAGED, NT>(tq, tk, tv, a, grid, st)
               : launch_tc_t<128, 0, PAGED, NT>(tq, tk, tv, a, grid, st);
  return f16 ? launch_tc_t<64, 1, PAGED, NT>(tq, tk, tv, a, grid, st)
             : launch_tc_t<64, 0, PAGED, NT>(tq, tk, tv, a, grid, st);
}

template <bool PAGED>
cudaError_t launch_tc(int nt, int D, int f16, const CUtensorMap& tq, const CUtensorMap& tk,
                      const CUtensorMap& tv, const AttnTcArgs& a, unsigned grid, cudaStream_t st) {
  return nt == 2 ? launch_tc_n<PAGED, 2>(D, f16, tq, tk, tv, a, grid, st)
                 : launch_tc_n<PAGED, 1>(D, f16, tq, tk, tv, a, grid, st);
}

template <int D, int F16>
cudaError_t launch_own_t(const OwnArgs& a, const JoinArgs& j, bool after_prefix, cudaStream_t st) {
  if (a.out) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(attn_own_kernel<D, F16, true>, own_smem<D>(), done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.n_rows * a.Hkv * a.mtiles * a.splits));
    cfg.blockDim = dim3(kOwnWarps * 32);
    cfg.dynamicSmemBytes = own_smem<D>();
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_own_kernel<D, F16, true>, a);
  }
  if (a.splits > 0) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(attn_own_kernel<D, F16, false>, own_smem<D>(), done);
    const unsigned grid = (unsigned)((long long)a.n_rows * a.Hkv * a.mtiles * a.splits);
    if (e == cudaSuccess)
      e = launch_ex(attn_own_kernel<D, F16, false>, dim3(grid), dim3(kOwnWarps * 32), own_smem<D>(), st,
                    after_prefix, a);
    if (e != cudaSuccess) return e;
  }
  // a warp per row and head once four would be more than 16 CTAs per SM
  const long long rows = (long long)j.n_rows * j.Hq;
  const bool pdl = after_prefix || a.splits > 0;
  if (rows > 16ll * sm_count())
    return launch_ex(attn_join_kernel<D, F16, 1>, dim3((unsigned)((rows + 3) / 4)),
                     dim3(kJoinThreads), 0, st, pdl, j);
  return launch_ex(attn_join_kernel<D, F16, 4>, dim3((unsigned)rows), dim3(kJoinThreads), 0, st,
                   pdl, j);
}

constexpr long long kAlonePositions = 2048;  // rows x prefix, see plan_prefix

// How m3_attn_prefix splits its work; the workspace follows from it.  It goes by
// the prefix's pages and the table's width: the rows' lengths live on the device.
struct PrefixPlan {
  int grp = 0, tpt = 0, nt = 0, units = 0;  // rows per row tile, row tiles of a CTA, such groups
  bool alone = false;                       // the prefix is read by every row for itself
  bool cluster = false;                     // and a row's splits join in a cluster
  int pre_splits = 0, pre_tiles = 0;     // splits of the prefix, key tiles of each
  int mtiles = 0, own_splits = 0;
  int64_t rows = 0, bytes = 0;
};

bool plan_prefix(int n_rows, int Hq, int Hkv, int D, int prefix_pages, int page, int max_pages,
                 PrefixPlan* p) {
  const int shift = page_shift(page);
  if (shift < 0 || n_rows < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 64 ||
      (D != 64 && D != 128) || prefix_pages < 0 || max_pages < 0)
    return false;
  const long long prefix = (long long)prefix_pages << shift, own = (long long)max_pages << shift;
  if (prefix > INT_MAX - 256 || own > INT_MAX - 256) return false;
  const int nsm = sm_count();
  p->grp = Hq / Hkv;
  p->tpt = kTile / p->grp;
  // Two row tiles per CTA from four pairs on (256 rows of 4 heads a KV head,
  // prefix 9000: 79.9 against 86.6 us with one; 1024 rows: 260 against 320).
  // Below, CTAs of one tile leave room for the rows' own positions beside them
  // (128 rows: 49.7 against 50.2)
  p->nt = n_rows >= 8 * p->tpt ? 2 : 1;
  p->units = (n_rows + p->nt * p->tpt - 1) / (p->nt * p->tpt);
  p->rows = (int64_t)n_rows * Hq;
  p->mtiles = (p->grp + 15) / 16;
  const long long key_tiles = (prefix + kTile - 1) / kTile;
  const long long ctas = (long long)n_rows * Hkv * p->mtiles;
  // splits into runs of 64 positions at least, for about four CTAs per SM
  auto small_splits = [&](long long positions, long long all) {
    long long s = (4ll * nsm * positions + all * ctas - 1) / (all * ctas);
    const long long most = (positions + 63) / 64;
    s = s > most ? most : s;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  };
  // A short prefix, or one row: every row reads it for itself, in one launch with
  // its own positions.  (Calls of 1 to 16 rows with prefixes of 128 to 4500, 40 own
  // positions, 32 heads on 8 of 128, in pages of 64, 256 and 1024: the two meet
  // between 2048 and 4096 rows x positions.  4 x 300 in pages of 256: 8.3 against
  // 12.4 us; 4 x 1024: 14.4 against 12.4; 16 x 300 in pages of 64: 16.0 against
  // 14.4; one row of 4500 with a table of 36 pages: 14.4 against 18.5.)
  p->alone = key_tiles > 0 && (n_rows == 1 || n_rows * prefix <= kAlonePositions);
  if (p->alone) {
    p->pre_splits = small_splits(prefix, prefix + own);
  } else if (key_tiles > 0) {
    // one round of CTAs over the SMs (a CTA fills one), whole key tiles
    long long s = nsm / ((long long)p->units * Hkv);
    s = s < 1 ? 1 : s > key_tiles ? key_tiles : s;
    s = s > kMaxParts - 64 ? kMaxParts - 64 : s;
    p->pre_tiles = (int)((key_tiles + s - 1) / s);
    p->pre_splits = (int)((key_tiles + p->pre_tiles - 1) / p->pre_tiles);
  }
  if (own > 0) p->own_splits = small_splits(own, p->alone ? prefix + own : own);
  // Few positions and rows: up to eight splits of 128 positions, which one cluster
  // joins in the same launch (4 rows, prefix 300: 6.3 against 7.7 us; with a table of
  // 36 pages of 256, which does not fit eight splits, 12.4 a call against 8.3)
  const long long small = (prefix + 127) / 128 + (own + 127) / 128;
  p->cluster = (p->alone || prefix == 0) && small > 0 && small <= kClusterMost && ctas * small <= 4ll * nsm;
  if (p->cluster) {
    p->pre_splits = (int)((prefix + 127) / 128);
    p->own_splits = (int)((own + 127) / 128);
  }
  const int64_t parts = p->pre_splits + p->own_splits;
  p->bytes = ((parts * p->rows * 8 + 15) & ~(int64_t)15) + parts * p->rows * D * 4;
  if (p->bytes == 0) p->bytes = 16;
  return p->rows <= INT_MAX && (long long)p->units * Hkv * p->pre_splits <= INT_MAX &&
         ctas * (p->own_splits + (p->alone ? p->pre_splits : 0)) <= INT_MAX;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// Strides of a [n][heads][D] operand: positive multiples of 8 elements.
bool good_strides(int64_t a, int64_t b) {
  return a > 0 && b > 0 && a % 8 == 0 && b % 8 == 0 && a < (1ll << 38) && b < (1ll << 38);
}

}  // namespace

}  // namespace m3

using namespace m3;

#define OPS_CK(call)                                                                  \
  do {                                                                                \
    const cudaError_t e_ = (call);                                                    \
    if (e_ != cudaSuccess)                                                            \
      return set_error(M3_ECUDA, std::string(#call) + ": " + cudaGetErrorString(e_)); \
  } while (0)

int m3::attn_prompt(int dtype, int n_seq, int n_q, int n_k, int Hq, int Hkv, int D, const void* q,
                    int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                    int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                    const int32_t* cu_q, const int32_t* cu_k, float scale, void* out,
                    int64_t o_token, int64_t o_head, float* lse, int* err, void* cuda_stream) {
  if (dtype != M3_KV_BF16 && dtype != M3_KV_F16) return set_error(M3_EINVAL, "dtype");
  if (n_seq < 0 || n_seq > 8192) return set_error(M3_EINVAL, "n_seq out of 0..8192");
  if (n_q < 0 || n_k < 0) return set_error(M3_EINVAL, "negative count");
  if (D != 64 && D != 128) return set_error(M3_EINVAL, "D: 64 or 128");
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 64)
    return set_error(M3_EINVAL, "Hq: a multiple of Hkv, up to 64 times it");
  if (!cu_k && n_k != n_q) return set_error(M3_EINVAL, "without cu_k, n_k is n_q");
  if (!(scale > 0.0f) || scale > 1e30f) return set_error(M3_EINVAL, "scale: positive");
  if (n_seq == 0 || n_q == 0) return M3_OK;
  if (!q || !out || !cu_q || (n_k && (!k || !v))) return set_error(M3_EINVAL, "null argument");
  if (!aligned16(q) || !aligned16(out) || !aligned16(k) || !aligned16(v))
    return set_error(M3_EINVAL, "q, k, v and out have to be 16-byte aligned");
  if (!good_strides(q_token, q_head) || !good_strides(o_token, o_head) ||
      (n_k && (!good_strides(k_token, k_head) || !good_strides(v_token, v_head))))
    return set_error(M3_EINVAL, "strides: positive multiples of 8 elements");
  const int f16 = dtype == M3_KV_F16;
  AttnTcArgs a{};
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.n_seq = n_seq;
  a.n_q = n_q;
  a.n_k = n_k;
  a.out = static_cast<uint16_t*>(out);
  a.o_token = o_token;
  a.o_head = o_head;
  a.lse = lse;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_token = q_token;
  a.q_head = q_head;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.err = err;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.grp = Hq / Hkv;
  a.tpt = kTile / a.grp;
  a.c = scale * kLog2e;
  CUtensorMap tq, tk, tv;
  bool ok = make_rows_map(&tq, f16, q, n_q, Hq, D, q_token, q_head, a.grp, a.tpt);
  // no key at all: the kernel reads none, any valid map will do
  ok = ok && make_rows_map(&tk, f16, n_k ? k : q, n_k ? n_k : n_q, n_k ? Hkv : Hq, D,
                           n_k ? k_token : q_token, n_k ? k_head : q_head, 1, kTile);
  ok = ok && make_rows_map(&tv, f16, n_k ? v : q, n_k ? n_k : n_q, n_k ? Hkv : Hq, D,
                           n_k ? v_token : q_token, n_k ? v_head : q_head, 1, kTile);
  if (!ok) return set_error(M3_EINVAL, "no tensor map for these strides");
  // every sequence's last unit may be short: at most one more unit each
  auto most = [&](int nt) { return n_q / (nt * a.tpt) + (n_seq < n_q ? n_seq : n_q); };
  // one row tile per CTA while there is an SM for each
  const int nt = (long long)most(1) * Hkv <= sm_count() ? 1 : 2;
  const long long units = most(nt);
  if (units * Hkv > INT_MAX) return set_error(M3_EINVAL, "too many tokens");
  OPS_CK(launch_tc<false>(nt, D, f16, tq, tk, tv, a, (unsigned)(units * Hkv),
                          static_cast<cudaStream_t>(cuda_stream)));
  return M3_OK;
}

extern "C" int m3_attn_prompt(int dtype, int n_seq, int n_q, int n_k, int Hq, int Hkv, int D,
                              const void* q, int64_t q_token, int64_t q_head, const void* k,
                              int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                              int64_t v_head, const int32_t* cu_q, const int32_t* cu_k,
                              float scale, void* out, int64_t o_token, int64_t o_head, float* lse,
                              void* cuda_stream) {
  return attn_prompt(dtype, n_seq, n_q, n_k, Hq, Hkv, D, q, q_token, q_head, k, k_token, k_head, v,
                     v_token, v_head, cu_q, cu_k, scale, out, o_token, o_head, lse, nullptr,
                     cuda_stream);
}

extern "C" int64_t m3_attn_prefix_workspace(int n_rows, int Hq, int Hkv, int D, int prefix_pages,
                                            int page, int max_pages) {
  PrefixPlan p;
  return plan_prefix(n_rows, Hq, Hkv, D, prefix_pages, page, max_pages, &p) ? p.bytes : 0;
}

extern "C" int m3_attn_prefix(int dtype, int n_rows, int Hq, int Hkv, int D, const void* q,
                              int64_t q_row, int64_t q_head, const void* pool, int n_pages,
                              int page, const int32_t* prefix_pages, int n_prefix_pages,
                              int prefix_len, const int32_t* table, int max_pages,
                              int64_t ld_table, const int32_t* lens, float scale, void* out,
                              int64_t o_row, int64_t o_head, float* lse, void* workspace,
                              int64_t workspace_bytes, void* cuda_stream) {
  if (dtype != M3_KV_BF16 && dtype != M3_KV_F16) return set_error(M3_EINVAL, "dtype");
  if (n_rows < 0 || n_pages < 0 || n_prefix_pages < 0 || prefix_len < 0 || max_pages < 0)
    return set_error(M3_EINVAL, "negative count");
  if (page_shift(page) < 0) return set_error(M3_EINVAL, "page: a power of two, 16..1024");
  if (D != 64 && D != 128) return set_error(M3_EINVAL, "D: 64 or 128");
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 64)
    return set_error(M3_EINVAL, "Hq: a multiple of Hkv, up to 64 times it");
  if ((long long)n_prefix_pages * page < prefix_len)
    return set_error(M3_EINVAL, "prefix_len is longer than prefix_pages");
  if (!(scale > 0.0f) || scale > 1e30f) return set_error(M3_EINVAL, "scale: positive");
  if (n_rows == 0) return M3_OK;
  if (ld_table < max_pages) return set_error(M3_EINVAL, "ld_table < max_pages");
  if (!q || !out || !lens || (max_pages && !table) || (prefix_len && !prefix_pages) ||
      (n_pages && !pool))
    return set_error(M3_EINVAL, "null argument");
  if (!aligned16(q) || !aligned16(out) || !aligned16(pool))
    return set_error(M3_EINVAL, "q, out and the pool have to be 16-byte aligned");
  if (!good_strides(q_row, q_head) || !good_strides(o_row, o_head))
    return set_error(M3_EINVAL, "strides: positive multiples of 8 elements");
  PrefixPlan p;
  if (!plan_prefix(n_rows, Hq, Hkv, D, n_prefix_pages, page, max_pages, &p))
    return set_error(M3_EINVAL, "too many rows or pages");
  if (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)
    return set_error(M3_EINVAL, "workspace: m3_attn_prefix_workspace bytes, 16-byte aligned");
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int f16 = dtype == M3_KV_F16, shift = page_shift(page);
  // pages without a pool hold nothing
  if (n_pages == 0) prefix_len = 0;
  const int pre = prefix_len > 0 ? p.pre_splits : 0, own = n_pages > 0 ? p.own_splits : 0;
  const bool shared = pre > 0 && !p.alone;
  const int64_t parts = pre + own;
  float2* ml = static_cast<float2*>(workspace);
  float* po = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       ((parts * p.rows * 8 + 15) & ~(int64_t)15));
  if (shared) {
    AttnTcArgs a{};
    a.pages = prefix_pages;
    a.n_prefix_pages = n_prefix_pages;
    a.n_pages = n_pages;
    a.shift = shift;
    a.prefix_len = prefix_len;
    a.n_rows = n_rows;
    a.splits = pre;
    a.tiles_per_split = p.pre_tiles;
    a.part_o = po;
    a.part_ml = ml;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.grp = p.grp;
    a.tpt = p.tpt;
    a.c = scale * kLog2e;
    CUtensorMap tq, tk;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)2 * Hkv,
                                (cuuint64_t)n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)page * D * 2,
                                   (cuuint64_t)page * D * 4 * Hkv};
    const cuuint32_t box[4] = {64, (cuuint32_t)(page < kTile ? page : kTile), 1, 1};
    if (!make_rows_map(&tq, f16, q, n_rows, Hq, D, q_row, q_head, a.grp, a.tpt) ||
        !make_map(&tk, f16, 4, pool, dims, strides, box))
      return set_error(M3_EINVAL, "no tensor map for these strides");
    OPS_CK(launch_tc<true>(p.nt, D, f16, tq, tk, tk, a, (unsigned)(p.units * Hkv * pre), st));
  }
  OwnArgs o{};
  o.q = static_cast<const uint16_t*>(q);
  o.q_row = q_row;
  o.q_head = q_head;
  o.pool = static_cast<const uint16_t*>(pool);
  o.table = table;
  o.ld_table = ld_table;
  o.lens = lens;
  o.n_pages = n_pages;
  o.shift = shift;
  o.max_pages = max_pages;
  o.n_rows = n_rows;
  o.Hq = Hq;
  o.Hkv = Hkv;
  o.grp = p.grp;
  o.mtiles = p.mtiles;
  o.prefix_pages = prefix_pages;
  o.prefix_len = prefix_len;
  o.pre_splits = shared ? 0 : pre;
  o.splits = own + o.pre_splits;
  o.c = scale * kLog2e;
  o.part_o = po + (int64_t)(pre - o.pre_splits) * p.rows * D;
  o.part_ml = ml + (int64_t)(pre - o.pre_splits) * p.rows;
  JoinArgs j{po, ml, lens, static_cast<uint16_t*>(out), o_row, o_head, lse, n_rows, Hq, (int)parts};
  if (p.cluster && o.splits > 0) {
    o.out = static_cast<uint16_t*>(out);
    o.o_row = o_row;
    o.o_head = o_head;
    o.lse = lse;
  }
  if (D == 128)
    OPS_CK(f16 ? (launch_own_t<128, 1>(o, j, shared, st)) : (launch_own_t<128, 0>(o, j, shared, st)));
  else
    OPS_CK(f16 ? (launch_own_t<64, 1>(o, j, shared, st)) : (launch_own_t<64, 0>(o, j, shared, st)));
  return M3_OK;
}

extern "C" int m3_ops_sync_status(void* cuda_stream) {
  OPS_CK(cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)));
  int e = 0;
  OPS_CK(cudaMemcpyFromSymbol(&e, g_ops_err, sizeof(int)));
  if (e == kErrNone) return M3_OK;
  const int zero = 0;
  OPS_CK(cudaMemcpyToSymbol(g_ops_err, &zero, sizeof(int)));
  return set_error(e == kErrTimeout ? M3_ETIMEOUT : M3_EDEVICE,
                   e == kErrTimeout ? "a device wait gave up" : "a kernel recorded an error");
}
