// ops.cu -- the serving operators of include/m3_ops.h that move and count:
// page tables and slot maps, the K/V store, rules on logits.  The attention
// operators are in ops_attn.cu.
#include <cuda_runtime.h>

#include <climits>
#include <string>

#include "common.cuh"
#include "launch.cuh"
#include "m3_ops.h"
#include "ops.cuh"

namespace m3 {

namespace {

// ------------------------------------------------------------------- map ---
// Every CTA scans the request lengths by itself (8 + 4 bytes a request, at
// most 96 KB from L2), so the map is one launch without a wait between CTAs:
// the table columns that the scan gives out are written by one CTA and read by
// none, since a token's page is taken from the free list by the same sum.
// The columns of the cached tokens are read only.  Bound by its few dependent
// reads: 4.4 us for 16 requests, 5.4 us for 256 with 109000 tokens (1.8 MB).
constexpr int kMapThreads = 512;
constexpr int kMapMaxReq = 8192;

struct MapArgs {
  const int32_t *fresh, *cached, *free_pages, *free_at;
  int32_t* table;
  int32_t *cu, *positions, *seqs, *lens, *taken;
  int64_t* slots;
  int64_t ld_table;
  int n_req, n_free, max_pages, shift, n_pages, start, n_tokens;
};

__device__ __forceinline__ int sat(long long v) { return v > INT_MAX ? INT_MAX : (int)v; }

__device__ __forceinline__ int free_page(const MapArgs& a, long long i) {
  if (i < 0 || i >= a.n_free) return -1;
  const int p = a.free_pages[i];
  return p >= 0 && p < a.n_pages ? p : -1;
}

__global__ void __launch_bounds__(kMapThreads) kv_map_kernel(const MapArgs a) {
  extern __shared__ int map_smem[];
  int* scu = map_smem;                // [n_req + 1] first token of each request
  int* soff = map_smem + a.n_req + 1;  // [n_req] pages given out before it
  __shared__ long long warp_tok[kMapThreads / 32], warp_pg[kMapThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int p1 = (1 << a.shift) - 1;
  // each thread's run of requests, then a scan over the threads (64-bit sums)
  const int per = (a.n_req + kMapThreads - 1) / kMapThreads;
  const int r0 = min(a.n_req, tid * per), r1 = min(a.n_req, r0 + per);
  auto load = [&](int r, int& f, int& c, int& want) {
    f = max(0, a.fresh[r]);
    c = a.cached ? max(0, a.cached[r]) : 0;
    const long long have = ((long long)c + p1) >> a.shift;
    const long long need = ((long long)c + f + p1) >> a.shift;
    want = (int)max(0ll, min(need, (long long)a.max_pages) - have);
  };
  long long tok = 0, pg = 0;
  for (int r = r0; r < r1; ++r) {
    int f, c, w;
    load(r, f, c, w);
    tok += f;
    pg += w;
  }
  long long it = tok, ip = pg;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(~0u, it, o), p = __shfl_up_sync(~0u, ip, o);
    if (lane >= o) {
      it += t;
      ip += p;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = it;
    warp_pg[warp] = ip;
  }
  __syncthreads();
  long long bt = it - tok, bp = ip - pg, all_tok = 0, all_pg = 0;
  for (int w = 0; w < kMapThreads / 32; ++w) {
    if (w < warp) {
      bt += warp_tok[w];
      bp += warp_pg[w];
    }
    all_tok += warp_tok[w];
    all_pg += warp_pg[w];
  }
  for (int r = r0; r < r1; ++r) {
    int f, c, w;
    load(r, f, c, w);
    scu[r] = sat(bt);
    soff[r] = sat(bp);
    bt += f;
    bp += w;
    if (blockIdx.x == 0) {
      a.cu[r] = scu[r];
      a.lens[r] = sat((long long)c + f);
    }
  }
  if (tid == 0) {
    scu[a.n_req] = sat(all_tok);
    if (blockIdx.x == 0) {
      a.cu[a.n_req] = sat(all_tok);
      *a.taken = sat(all_pg);
    }
  }
  __syncthreads();
  const int first = a.free_at ? max(0, *a.free_at) : 0;

  // the new table columns: one warp per request
  const int nwarps = gridDim.x * (kMapThreads / 32);
  for (int r = blockIdx.x * (kMapThreads / 32) + warp; r < a.n_req; r += nwarps) {
    int f, c, w;
    load(r, f, c, w);
    if (w == 0) continue;
    int32_t* row = a.table + r * a.ld_table + (((long long)c + p1) >> a.shift);
    for (int i = lane; i < w; i += 32) row[i] = free_page(a, (long long)first + soff[r] + i);
  }

  // the tokens: four in a row per thread, so that the three maps leave in
  // 16-byte stores
  const int total = min(scu[a.n_req], a.n_tokens);
  const long long step = 4ll * gridDim.x * kMapThreads;
  for (long long t0 = 4ll * (blockIdx.x * kMapThreads + tid); t0 < a.n_tokens; t0 += step) {
    int pos[4], seq[4];
    long long slot[4];
    int lo = 0;
    if (t0 < total) {  // the last request that starts at or before t0
      int hi = a.n_req - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (scu[mid] <= t0) lo = mid;
        else hi = mid - 1;
      }
    }
    int of = -1, f = 0, c = 0, w = 0;  // the request whose lengths are loaded
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = t0 + i;
      pos[i] = seq[i] = -1;
      slot[i] = -1;
      if (t >= total) continue;
      while (scu[lo + 1] <= t) ++lo;
      if (lo != of) {
        load(lo, f, c, w);
        of = lo;
      }
      const long long j = (long long)c + (t - scu[lo]);  // place in the request's table
      seq[i] = lo;
      pos[i] = sat(a.start + j);
      const long long col = j >> a.shift, have = ((long long)c + p1) >> a.shift;
      int page = -1;
      if (col < a.max_pages) {
        if (col >= have) {
          page = free_page(a, (long long)first + soff[lo] + (col - have));
        } else {
          page = a.table[lo * a.ld_table + col];
          if (page >= a.n_pages) page = -1;
        }
      }
      if (page >= 0) slot[i] = ((long long)page << a.shift) | (j & p1);
    }
    if (t0 + 4 <= a.n_tokens) {
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.seqs + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < a.n_tokens) {
          a.positions[t0 + i] = pos[i];
          a.seqs[t0 + i] = seq[i];
          a.slots[t0 + i] = slot[i];
        }
    }
  }
}

// ----------------------------------------------------------------- store ---
// 16-byte pieces: a thread keeps one (K or V, head, piece) column and walks
// tokens, four loads in flight; VEC = false: sources whose rows are not
// 16-byte aligned, read in 16-bit words.  Bound by HBM: 16387 tokens of 8 KV heads
// of 128 (134 MB) in 23.4 us, 5.7 TB/s; 16 tokens in 1.7 us.
constexpr int kStoreThreads = 256;
constexpr int kStoreUnroll = 4;

struct StoreArgs {
  const uint16_t *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  const int64_t* slots;
  uint4* pool;
  long long n_slots;
  int n_tokens, Hkv, pieces, shift;
};

template <bool VEC>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(const StoreArgs a) {
  const int ncol = 2 * a.Hkv * a.pieces;
  // threads of a block: `groups` tokens side by side, each over the columns
  const int width = min(ncol, kStoreThreads), groups = kStoreThreads / width;
  const int g = threadIdx.x / width;
  if (g >= groups) return;
  const long long page_pieces = (long long)ncol << a.shift;
  for (int col = threadIdx.x % width; col < ncol; col += width) {
    const int hv = col / a.pieces, piece = col % a.pieces;  // head slot (K heads, V heads)
    const bool isv = hv >= a.Hkv;
    const uint16_t* src = isv ? a.v + (hv - a.Hkv) * a.v_head : a.k + hv * a.k_head;
    const int64_t st = isv ? a.v_token : a.k_token;
    const long long step = (long long)gridDim.x * groups;
    for (long long t0 = (long long)blockIdx.x * groups + g; t0 < a.n_tokens;
         t0 += step * kStoreUnroll) {
      uint4 val[kStoreUnroll];
      long long slot[kStoreUnroll];
#pragma unroll
      for (int u = 0; u < kStoreUnroll; ++u) {
        const long long t = t0 + u * step;
        slot[u] = -1;
        if (t < a.n_tokens) {
          slot[u] = __ldg(a.slots + t);
          const uint16_t* p = src + t * st + piece * 8;  // read whatever the slot says
          if constexpr (VEC) {
            val[u] = __ldg(reinterpret_cast<const uint4*>(p));
          } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
            val[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (slot[u] >= a.n_slots) slot[u] = -1;
        }
      }
#pragma unroll
      for (int u = 0; u < kStoreUnroll; ++u)
        if (slot[u] >= 0) {
          const long long page = slot[u] >> a.shift, off = slot[u] & ((1ll << a.shift) - 1);
          a.pool[page * page_pieces + (((long long)hv << a.shift) + off) * a.pieces + piece] =
              val[u];
        }
    }
  }
}

// ----------------------------------------------------------------- rules ---
// A CTA takes a run of one row's vocabulary.  It asks for everything it will
// need at once -- its logits, the mask's words, the history, the biases -- then
// notes in one word of shared memory per token how often the row's history has
// it and whether a bias, or several, name it (additions and flags: the order of
// the atomics does not matter).  Meanwhile the logits are written out under the
// mask alone: few tokens have a word other than 0, and those are taken up again
// afterwards, from a list, where the mask has left them as they were.  (Rules
// inside the streaming loop bind the kernel by its instructions.)  Every run of
// a row reads the whole history again, so runs are long.  2 x 16385 fp32 with
// 1500 tokens of history: 4.4 us, bound by the chain of its reads.
constexpr int kRuleThreads = 512;
constexpr int kRuleRun = 8192;  // logits of the longest run
constexpr int kBiased = 1 << 30;  // of the word: a bias names the token; below them the count
constexpr int kSeveral = 1 << 29;  // several do
constexpr uint16_t kNoToken = 0xFFFF;
constexpr int kRuleMaxBias = 4096, kRuleMaxHistory = 1 << 24;  // counts are exact in fp32

// x plus the biases of a token in their order, among the entries from..n - 1:
// a warp's work, 128 entries at a time.  For tokens that several entries name;
// one with a single entry has it at hand.
template <typename Token, typename Bias>
__device__ __forceinline__ float add_biases(float x, int token, int from, int n, int lane,
                                            Token token_of, Bias bias_of) {
  for (int b = from; b < n; b += 128) {
    bool is[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = b + 32 * q + lane;
      is[q] = e < n && token_of(e) == token;
    }
    if (!__any_sync(~0u, is[0] || is[1] || is[2] || is[3])) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v = is[q] ? bias_of(b + 32 * q + lane) : 0.0f;
      for (unsigned m = __ballot_sync(~0u, is[q]); m; m &= m - 1)
        x += __shfl_sync(~0u, v, __ffs(m) - 1);
    }
  }
  return x;
}

// atom.shared as it stands: the compiler's own form for a counter gathers the
// warp's lanes first, some 20 instructions at each place it is used.
__device__ __forceinline__ int smem_add(int* p, int v) {
  int old;
  asm volatile("atom.shared.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(smem_u32(p)), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ int smem_or(int* p, int v) {
  int old;
  asm volatile("atom.shared.or.b32 %0, [%1], %2;" : "=r"(old) : "r"(smem_u32(p)), "r"(v) : "memory");
  return old;
}

struct RuleArgs {
  const void* in;
  void* out;
  int64_t ld_in, ld_out;
  const int32_t* history;
  int64_t ld_history;
  const int32_t* hist_len;
  const float *rep, *freq, *pres;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* mask;
  const int32_t* mask_row;
  int vocab, n_history, n_bias, n_masks, words, run, runs;
  int parts, range, slots;  // of logit_touch_kernel
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

__device__ __forceinline__ bool allows(const uint32_t* mask, int at) {
  return !mask || ((__ldg(mask + (at >> 5)) >> (at & 31)) & 1);
}
// A logit under the penalties, its token c times in the history.
__device__ __forceinline__ float penalise(float x, int c, float rep, float freq, float pres) {
  if (c > 0) {
    x = x > 0.0f ? x / rep : x * rep;
    x -= freq * (float)c;
    x -= pres;
  }
  return x;
}

// What a CTA of logit_rules_kernel has noted, in shared memory.
struct RuleNotes {
  const int* note;       // [run]
  const uint16_t* list;  // tokens noted, from s0
  int n_list;
  uint16_t* named;       // [n_bias] the biases' tokens
  float* bias;           // [n_bias]
  int n_bias;
  int* warp_sum;         // [warps]
};

// The tokens that several biases name: those entries side by side, in their
// order, then a warp per token looks through them.  Out of line, since few calls
// have such tokens and the rest of the kernel wants the registers.  4096 biases
// on 80 x 8192 logits: 21 us a call with a token each, 188 all of one token, 945
// two to a token; on 2 x 16385: 10, 178 and 19.
template <typename T>
__device__ __noinline__ void finish_several(const RuleNotes r, const T* in, T* out, long long s0,
                                            const uint32_t* mask, float rep, float freq, float pres) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kEach = kRuleMaxBias / kRuleThreads;  // entries of a thread, in a row
  const int per = (r.n_bias + kRuleThreads - 1) / kRuleThreads;
  uint16_t token[kEach];
  float value[kEach];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = tid * per + i;
    token[i] = i < per && e < r.n_bias ? r.named[e] : kNoToken;
    if (token[i] != kNoToken && !(r.note[token[i]] & kSeveral)) token[i] = kNoToken;
    value[i] = token[i] != kNoToken ? r.bias[e] : 0.0f;
    mine += token[i] != kNoToken;
  }
  int place = mine;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, place, o);
    if (lane >= o) place += v;
  }
  if (lane == 31) r.warp_sum[warp] = place;
  __syncthreads();  // (every thread has its entries in registers)
  int n_several = 0;
  place -= mine;
  for (int w = 0; w < kRuleThreads / 32; ++w) {
    if (w < warp) place += r.warp_sum[w];
    n_several += r.warp_sum[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (token[i] != kNoToken) {
      r.named[place] = token[i];
      r.bias[place++] = value[i];
    }
  __syncthreads();
  for (int k = warp; k < r.n_list; k += kRuleThreads / 32) {
    const int w = r.note[r.list[k]], at = (int)(s0 + r.list[k]);
    if (!(w & kSeveral) || !allows(mask, at)) continue;
    const float x = add_biases(
        penalise(to_f(in[at]), w & (kSeveral - 1), rep, freq, pres), r.list[k], 0, n_several, lane,
        [&](int e) { return r.named[e]; }, [&](int e) { return r.bias[e]; });
    if (lane == 0) out[at] = from_f<T>(x);
  }
}

template <typename T>
__global__ void __launch_bounds__(kRuleThreads, 3) logit_rules_kernel(const RuleArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int KV = kRuleRun / (VEC * kRuleThreads);  // 16-byte pieces per thread
  extern __shared__ __align__(16) int rule_smem[];  // cleared 16 bytes at a time
  const int tid = threadIdx.x;
  const int row = blockIdx.x / a.runs, part = blockIdx.x % a.runs;
  const T* in = static_cast<const T*>(a.in) + row * a.ld_in;
  T* out = static_cast<T*>(a.out) + row * a.ld_out;
  // runs start on a 16-byte boundary of the row, so the first may be short
  const int lead = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) % VEC);
  const bool vec_out = (reinterpret_cast<uintptr_t>(out) / sizeof(T)) % VEC == (unsigned)lead;
  const long long s0 = (long long)part * a.run - lead;
  const int lo = (int)max(s0, 0ll), hi = (int)min(s0 + a.run, (long long)a.vocab);
  if (lo >= hi) return;
  uint4 raw[KV];
#pragma unroll
  for (int u = 0; u < KV; ++u) {
    const int j = (u * kRuleThreads + tid) * VEC;
    if (j < a.run && s0 + j >= lo && s0 + j + VEC <= hi)
      raw[u] = *reinterpret_cast<const uint4*>(in + s0 + j);
  }
  const float rep = a.rep ? __ldg(a.rep + row) : 1.0f, freq = a.freq ? __ldg(a.freq + row) : 0.0f;
  const float pres = a.pres ? __ldg(a.pres + row) : 0.0f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_row ? __ldg(a.mask_row + row) : (a.n_masks == 1 ? 0 : row);
    if (m >= 0 && m < a.n_masks) mask = a.mask + (size_t)m * a.words;
  }
  uint32_t mbits[KV];
#pragma unroll
  for (int u = 0; u < KV; ++u) {
    const long long i0 = s0 + (u * kRuleThreads + tid) * VEC;
    mbits[u] = mask && i0 >= lo && i0 < hi ? __ldg(mask + (i0 >> 5)) : 0u;
  }
  const bool counts = a.history != nullptr, biases = a.n_bias > 0, noted = counts || biases;
  const int32_t* hist = a.history + (counts ? row * a.ld_history : 0);
  const bool hvec = counts && (reinterpret_cast<uintptr_t>(hist) & 15) == 0;
  int n_hist = a.n_history;
  int4 h0 = make_int4(-1, -1, -1, -1), h1 = h0;  // the first of the history
  if (hvec) {
    if (tid < n_hist >> 2) h0 = __ldg(reinterpret_cast<const int4*>(hist) + tid);
    if (tid + kRuleThreads < n_hist >> 2)
      h1 = __ldg(reinterpret_cast<const int4*>(hist) + tid + kRuleThreads);
  }
  if (counts && a.hist_len) n_hist = min(n_hist, max(0, __ldg(a.hist_len + row)));
  const int32_t* ids = a.bias_ids + (size_t)row * a.n_bias;
  const float* val = a.bias + (size_t)row * a.n_bias;
  int id0 = -1;
  float val0 = 0.0f;
  if (tid < a.n_bias) {
    id0 = __ldg(ids + tid);
    val0 = __ldg(val + tid);
  }
  int* note = rule_smem;                                    // [run]
  // the biases and their tokens, counted from s0 (kNoToken: outside the run)
  float* bias = reinterpret_cast<float*>(rule_smem + a.run);       // [n_bias]
  uint16_t* named = reinterpret_cast<uint16_t*>(bias + a.n_bias);  // [n_bias]
  uint16_t* list = named + a.n_bias;  // [run] tokens noted, from s0
  __shared__ int n_list, several, warp_sum[kRuleThreads / 32];
  if (noted) {
    if (tid == 0) n_list = several = 0;
    for (int i = tid * 4; i < a.run; i += kRuleThreads * 4)
      *reinterpret_cast<int4*>(note + i) = make_int4(0, 0, 0, 0);
    __syncthreads();
  }
  if (counts) {
    const unsigned span = (unsigned)(hi - lo);
    auto add = [&](int id) {
      if ((unsigned)id - (unsigned)lo >= span) return;
      const int at = (int)(id - s0);
      if (smem_add(&note[at], 1) == 0) list[smem_add(&n_list, 1)] = (uint16_t)at;
    };
    auto add4 = [&](int i, int4 v) {
      if (4 * i + 4 > n_hist) {  // the last piece: places past the end name no token
        v.x = 4 * i < n_hist ? v.x : -1;
        v.y = 4 * i + 1 < n_hist ? v.y : -1;
        v.z = 4 * i + 2 < n_hist ? v.z : -1;
        v.w = -1;
      }
      add(v.x);
      add(v.y);
      add(v.z);
      add(v.w);
    };
    int done = 0;
    if (hvec) {
      add4(tid, h0);
      add4(tid + kRuleThreads, h1);
      const int had = min(8 * kRuleThreads, a.n_history & ~3);  // places h0 and h1 cover
      for (int i = had / 4 + tid; i < n_hist >> 2; i += kRuleThreads)
        add4(i, __ldg(reinterpret_cast<const int4*>(hist) + i));
      done = max(had, n_hist & ~3);
    }
    for (int i = done + tid; i < n_hist; i += kRuleThreads) add(__ldg(hist + i));
  }
  if (biases) {
    auto name = [&](int e, int id, float b) {
      const bool ours = id >= lo && id < hi;
      const int at = (int)(id - s0);
      named[e] = ours ? (uint16_t)at : kNoToken;
      bias[e] = b;
      if (!ours) return;
      const int was = smem_or(&note[at], kBiased);
      if (was == 0) list[smem_add(&n_list, 1)] = (uint16_t)at;
      if (was & kBiased) {
        smem_or(&note[at], kSeveral);
        several = 1;
      }
    };
    if (tid < a.n_bias) name(tid, id0, val0);
    for (int e = tid + kRuleThreads; e < a.n_bias; e += kRuleThreads)
      name(e, __ldg(ids + e), __ldg(val + e));
  }

  // the run under the mask alone
#pragma unroll
  for (int u = 0; u < KV; ++u) {
    const int j = (u * kRuleThreads + tid) * VEC;
    const long long i0 = s0 + j;
    if (j < a.run && i0 >= lo && i0 + VEC <= hi) {
      T x[VEC];
      *reinterpret_cast<uint4*>(x) = raw[u];
      if (mask) {
        const int sh = (int)(i0 & 31);
        const uint32_t w1 = sh + VEC > 32 ? __ldg(mask + (i0 >> 5) + 1) : 0u;
        const uint32_t bits = __funnelshift_r(mbits[u], w1, sh);  // of i0, i0 + 1, ...
#pragma unroll
        for (int q = 0; q < VEC; ++q)
          if (!((bits >> q) & 1)) x[q] = from_f<T>(-INFINITY);
      }
      if (vec_out) {
        *reinterpret_cast<uint4*>(out + i0) = *reinterpret_cast<const uint4*>(x);
      } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) out[i0 + q] = x[q];
      }
    }
  }
  auto allowed = [&](int at) { return allows(mask, at); };
  // its first and last few, where a 16-byte piece reaches past it
  const int head = (int)min((long long)hi, s0 + (lo - s0 + VEC - 1) / VEC * VEC);
  const int tail = (int)max((long long)head, s0 + (hi - s0) / VEC * VEC);
  if (tid < (head - lo) + (hi - tail)) {
    const int at = tid < head - lo ? lo + tid : tail + (tid - (head - lo));
    out[at] = allowed(at) ? in[at] : from_f<T>(-INFINITY);
  }
  if (!noted) return;
  __syncthreads();  // the notes are complete, and what this CTA wrote is there

  // (a noted token's logit comes from L1; out's, where that is logits, is the same)
  auto penalised = [&](int at, int w) {
    return penalise(to_f(in[at]), w & (kSeveral - 1), rep, freq, pres);
  };
  for (int k = tid; k < n_list; k += kRuleThreads) {  // those without a bias
    const int w = note[list[k]], at = (int)(s0 + list[k]);
    if (!(w & kBiased) && allowed(at)) out[at] = from_f<T>(penalised(at, w));
  }
  if (!biases) return;
  for (int e = tid; e < a.n_bias; e += kRuleThreads) {  // with one
    if (named[e] == kNoToken) continue;
    const int w = note[named[e]], at = (int)(s0 + named[e]);
    if (!(w & kSeveral) && allowed(at)) out[at] = from_f<T>(penalised(at, w) + bias[e]);
  }
  if (!several) return;
  finish_several<T>(RuleNotes{note, list, n_list, named, bias, a.n_bias, warp_sum}, in, out, s0, mask, rep,
                    freq, pres);
}

// The same in two launches, for logits that fill the GPU several times over:
// there the waits of a run's history, between its loads and its stores, leave
// HBM idle.  (Us a call in one launch and in two, 4096 tokens of history and 300
// biases: 192 x 200000 93 and 86 in fp32, 74 and 58 in 16 bits; 80 x 200000 44 and
// 37, 33 and 27; 64 x 200000, which stays in one, 35 and 31, 27 and 26; 192 x 50000
// 33 and 36, 28 and 33; 64 x 50000 15 and 20, 13 and 19.)  The first streams the
// logits under the mask alone, with nothing to wait for; the second takes up a
// row's noted tokens, kept in a hash table in shared memory that it builds while
// the first one ends.
constexpr int kMaskThreads = 256;
constexpr int kMaskPieces = 4;

template <typename T>
__global__ void __launch_bounds__(kMaskThreads) logit_mask_kernel(const RuleArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  pdl_launch_dependents();
  const int tid = threadIdx.x, row = blockIdx.x / a.runs, part = blockIdx.x % a.runs;
  const T* in = static_cast<const T*>(a.in) + row * a.ld_in;
  T* out = static_cast<T*>(a.out) + row * a.ld_out;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_row ? __ldg(a.mask_row + row) : (a.n_masks == 1 ? 0 : row);
    if (m >= 0 && m < a.n_masks) mask = a.mask + (size_t)m * a.words;
  }
  if (!mask && in == out) return;
  const int lead = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) % VEC);
  const bool vec_out = (reinterpret_cast<uintptr_t>(out) / sizeof(T)) % VEC == (unsigned)lead;
  const long long s0 = (long long)part * a.run - lead;
  const int lo = (int)max(s0, 0ll), hi = (int)min(s0 + a.run, (long long)a.vocab);
  uint4 raw[kMaskPieces];
  uint32_t word[kMaskPieces];
#pragma unroll
  for (int u = 0; u < kMaskPieces; ++u) {
    const long long i0 = s0 + (u * kMaskThreads + tid) * VEC;
    const bool whole = i0 >= lo && i0 + VEC <= hi;
    if (whole) raw[u] = *reinterpret_cast<const uint4*>(in + i0);
    word[u] = mask && whole ? __ldg(mask + (i0 >> 5)) : ~0u;
  }
#pragma unroll
  for (int u = 0; u < kMaskPieces; ++u) {
    const long long i0 = s0 + (u * kMaskThreads + tid) * VEC;
    if (i0 < lo || i0 + VEC > hi) continue;
    T x[VEC];
    *reinterpret_cast<uint4*>(x) = raw[u];
    if (mask) {
      const int sh = (int)(i0 & 31);
      const uint32_t w1 = sh + VEC > 32 ? __ldg(mask + (i0 >> 5) + 1) : 0u;
      const uint32_t bits = __funnelshift_r(word[u], w1, sh);
#pragma unroll
      for (int q = 0; q < VEC; ++q)
        if (!((bits >> q) & 1)) x[q] = from_f<T>(-INFINITY);
    }
    if (vec_out) {
      *reinterpret_cast<uint4*>(out + i0) = *reinterpret_cast<const uint4*>(x);
    } else {
#pragma unroll
      for (int q = 0; q < VEC; ++q) out[i0 + q] = x[q];
    }
  }
  // the run's first and last few, where a 16-byte piece reaches past it
  const int head = (int)min((long long)hi, s0 + (lo - s0 + VEC - 1) / VEC * VEC);
  const int tail = (int)max((long long)head, s0 + (hi - s0) / VEC * VEC);
  if (tid < (head - lo) + (hi - tail)) {
    const int at = tid < head - lo ? lo + tid : tail + (tid - (head - lo));
    out[at] = !mask || ((__ldg(mask + (at >> 5)) >> (at & 31)) & 1) ? in[at]
                                                                   : from_f<T>(-INFINITY);
  }
}

constexpr int kTouchSlots = 16384;   // of the largest table
constexpr int kTouchTokens = 8192;   // it takes up to this many different tokens

inline size_t touch_smem(int slots, bool biases) {
  return (size_t)slots * (biases ? 12 : 8) + (size_t)kTouchTokens * 2;
}

constexpr int kTouchThreads = 1024;
constexpr int kAtOnce = 4;

template <typename T>
__global__ void __launch_bounds__(kTouchThreads, 1) logit_touch_kernel(const RuleArgs a) {
  extern __shared__ int touch_raw[];
  const int S = a.slots;
  int* key = touch_raw;       // [S] token, or -1
  int* cnt = key + S;         // [S] times in the history
  int* code = cnt + S;        // [S] n_bias - its first bias entry, or 0; kSeveral (with biases)
  const bool biases = a.n_bias > 0;
  uint16_t* list = reinterpret_cast<uint16_t*>(touch_raw + S * (biases ? 3 : 2));
  __shared__ int n_list;
  const int tid = threadIdx.x, row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int lo = part * a.range, hi = min(a.vocab, lo + a.range);
  const unsigned span = (unsigned)max(hi - lo, 0);
  const int shift = __clz(S - 1);
  const int32_t* ids = a.bias_ids + (size_t)row * a.n_bias;
  const float* val = a.bias + (size_t)row * a.n_bias;
  const int32_t* hist = a.history ? a.history + row * a.ld_history : nullptr;
  // asked for ahead of the table: the first of the history and of the biases
  int first[kAtOnce], n_hist = a.n_history;
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u)
    first[u] = hist && tid + u * kTouchThreads < n_hist ? __ldg(hist + tid + u * kTouchThreads) : -1;
  if (hist && a.hist_len) n_hist = min(n_hist, max(0, __ldg(a.hist_len + row)));
  const int id0 = tid < a.n_bias ? __ldg(ids + tid) : -1;
  for (int i = tid; i < S; i += kTouchThreads) {
    key[i] = -1;
    cnt[i] = 0;
    if (biases) code[i] = 0;
  }
  if (tid == 0) n_list = 0;
  __syncthreads();
  auto slot_of = [&](int id) -> int {
    int h = (int)(((unsigned)id * 2654435761u) >> shift);  // multiplicative hashing (Knuth)
    for (;;) {  // ends: each entry comes here once, and they are fewer than the slots
      const int was = atomicCAS(&key[h], -1, id);
      if (was == -1 || was == id) return h;
      h = (h + 1) & (S - 1);
    }
  };
  if (hist) {
    for (int i0 = tid; i0 < n_hist; i0 += kAtOnce * kTouchThreads) {  // several loads under way
      int id[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = i0 + u * kTouchThreads;
        id[u] = i >= n_hist ? -1 : i0 == tid ? first[u] : __ldg(hist + i);
      }
#pragma unroll 1
      for (int u = 0; u < kAtOnce; ++u) {
        const int v = u == 0 ? id[0] : u == 1 ? id[1] : u == 2 ? id[2] : id[3];
        if ((unsigned)v - (unsigned)lo < span) atomicAdd(&cnt[slot_of(v)], 1);
      }
    }
  }
  // The first entry of each token owns it, whatever the order of the atomics.
  // (4096 biases in place on 64 x 50000 logits: 26 us a call with a token each,
  // 223 all of one token, 530 two to a token.)
  int slot0 = 0;  // of the thread's first entry
  for (int e = tid; e < a.n_bias; e += kTouchThreads) {
    const int id = e == tid ? id0 : __ldg(ids + e);
    if ((unsigned)id - (unsigned)lo >= span) continue;
    const int h = slot_of(id);
    if (e == tid) slot0 = h;
    atomicMax(&code[h], a.n_bias - e);
  }
  __syncthreads();
  // and the others say that there are several
  for (int e = tid; e < a.n_bias; e += kTouchThreads) {
    const int id = e == tid ? id0 : __ldg(ids + e);
    if ((unsigned)id - (unsigned)lo >= span) continue;
    int h = e == tid ? slot0 : (int)(((unsigned)id * 2654435761u) >> shift);
    while (key[h] != id && key[h] >= 0) h = (h + 1) & (S - 1);
    // (an id read again that is not there, since somebody has written it
    // meanwhile, neither takes a slot nor counts)
    if (key[h] == id && (code[h] & ~kSeveral) != a.n_bias - e) atomicOr(&code[h], kSeveral);
  }
  // the taken slots side by side: one addition to the counter per warp (one per
  // token or per 32 slots, and they queue for it)
  int mine = 0;
  for (int i = tid; i < S; i += kTouchThreads) mine += key[i] >= 0;
  int place = mine;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, place, o);
    if ((tid & 31) >= o) place += v;
  }
  int base = 0;
  if ((tid & 31) == 31) base = smem_add(&n_list, place);
  place += __shfl_sync(~0u, base, 31) - mine;
  for (int i = tid; i < S; i += kTouchThreads)
    if (key[i] >= 0) list[place++] = (uint16_t)i;
  const float rep = a.rep ? __ldg(a.rep + row) : 1.0f, freq = a.freq ? __ldg(a.freq + row) : 0.0f;
  const float pres = a.pres ? __ldg(a.pres + row) : 0.0f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_row ? __ldg(a.mask_row + row) : (a.n_masks == 1 ? 0 : row);
    if (m >= 0 && m < a.n_masks) mask = a.mask + (size_t)m * a.words;
  }
  T* out = static_cast<T*>(a.out) + row * a.ld_out;
  __syncthreads();
  pdl_wait();  // the logits are there
  const int lane = tid & 31;
  for (int k0 = tid - lane; k0 < n_list; k0 += kAtOnce * kTouchThreads) {
    int h[kAtOnce];
    float y[kAtOnce];
    bool ok[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int k = k0 + lane + u * kTouchThreads;
      h[u] = list[min(k, n_list - 1)];
      const int at = key[h[u]];
      ok[u] = k < n_list && (!mask || ((__ldg(mask + (at >> 5)) >> (at & 31)) & 1));
      y[u] = to_f(__ldcg(out + at));
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int at = key[h[u]], c = cnt[h[u]];
      float x = penalise(y[u], c, rep, freq, pres);
      if (biases) {
        const int w = ok[u] ? code[h[u]] : 0, e = a.n_bias - (w & ~kSeveral);
        if (w > 0 && !(w & kSeveral)) x += __ldg(val + e);
        for (unsigned m = __ballot_sync(~0u, w & kSeveral); m; m &= m - 1) {
          const int from = __ffs(m) - 1;
          const float y = add_biases(
              __shfl_sync(~0u, x, from), __shfl_sync(~0u, at, from), __shfl_sync(~0u, e, from),
              a.n_bias, lane, [&](int f) { return __ldg(ids + f); },
              [&](int f) { return __ldg(val + f); });
          if (lane == from) x = y;
        }
      }
      if (ok[u]) out[at] = from_f<T>(x);
    }
  }
}

template <typename T>
cudaError_t launch_rules_two(RuleArgs a, int n_rows, bool stream_out, cudaStream_t st) {
  if (stream_out) {
    a.run = kMaskThreads * kMaskPieces * (16 / (int)sizeof(T));
    a.runs = (int)(((long long)a.vocab + 7 + a.run - 1) / a.run);
    logit_mask_kernel<T><<<(unsigned)(n_rows * a.runs), kMaskThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.history && !a.n_bias)) return e;
  }
  // a row's tokens in one table, or each table a part of the vocabulary
  const long long tokens = (long long)a.n_history + a.n_bias;
  a.parts = tokens <= kTouchTokens ? 1 : (a.vocab + kTouchTokens - 1) / kTouchTokens;
  a.range = (a.vocab + a.parts - 1) / a.parts;
  const long long most = tokens < a.range ? tokens : a.range;
  a.slots = 256;  // a quarter of the slots or more stays free
  while (a.slots * 3ll < most * 4) a.slots <<= 1;
  const size_t smem = touch_smem(a.slots, a.n_bias > 0);
  const cudaError_t e =
      cudaFuncSetAttribute(logit_touch_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)touch_smem(kTouchSlots, true));
  if (e != cudaSuccess) return e;
  return launch_ex(logit_touch_kernel<T>, dim3((unsigned)(n_rows * a.parts)), dim3(kTouchThreads),
                   smem, st, stream_out, a);
}

template <typename T>
cudaError_t launch_rules(const RuleArgs& a, int n_rows, cudaStream_t st) {
  if (a.parts) return launch_rules_two<T>(a, n_rows, a.in != a.out || a.mask, st);
  const size_t smem =
      a.history || a.n_bias ? 6 * ((size_t)a.run + a.n_bias) : 0;
  if (smem > 40 * 1024) {  // past the default limit with what the kernel holds itself
    const cudaError_t e =
        cudaFuncSetAttribute(logit_rules_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             6 * (kRuleRun + kRuleMaxBias));
    if (e != cudaSuccess) return e;
  }
  logit_rules_kernel<T><<<(unsigned)(n_rows * a.runs), kRuleThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int page_shift(int page) {
  if (page < 16 || page > 1024 || (page & (page - 1))) return -1;
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

int sm_count() {
  static thread_local int dev_of = -1, n = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev != dev_of) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    dev_of = dev;
  }
  return n;
}

}  // namespace m3

using namespace m3;

#define OPS_CK(call)                                                                  \
  do {                                                                                \
    const cudaError_t e_ = (call);                                                    \
    if (e_ != cudaSuccess)                                                            \
      return set_error(M3_ECUDA, std::string(#call) + ": " + cudaGetErrorString(e_)); \
  } while (0)

extern "C" int m3_kv_map(int n_req, const int32_t* fresh, const int32_t* cached,
                         const int32_t* free_pages, int n_free, const int32_t* free_at,
                         int32_t* table, int max_pages, int64_t ld_table, int page, int n_pages,
                         int start, int n_tokens, int32_t* cu, int32_t* positions, int64_t* slots,
                         int32_t* seqs, int32_t* lens, int32_t* taken, void* cuda_stream) {
  if (n_req < 1 || n_req > kMapMaxReq) return set_error(M3_EINVAL, "n_req out of 1..8192");
  const int shift = page_shift(page);
  if (shift < 0) return set_error(M3_EINVAL, "page: a power of two, 16..1024");
  if (n_free < 0 || max_pages < 0 || n_pages < 0 || n_tokens < 0 || start < 0)
    return set_error(M3_EINVAL, "negative count");
  if (ld_table < max_pages) return set_error(M3_EINVAL, "ld_table < max_pages");
  if (!fresh || !cu || !lens || !taken || (n_free && !free_pages) || (max_pages && !table) ||
      (n_tokens && (!positions || !slots || !seqs)))
    return set_error(M3_EINVAL, "null argument");
  // every CTA reads the inputs while others write
  struct Span {
    const void* p;
    size_t bytes;
  };
  const size_t n = n_req, nt = n_tokens;
  const Span ins[] = {{fresh, 4 * n}, {cached, 4 * n}, {free_pages, 4 * (size_t)n_free}, {free_at, 4}};
  const Span outs[] = {{cu, 4 * (n + 1)}, {lens, 4 * n},  {taken, 4},
                       {positions, 4 * nt}, {seqs, 4 * nt}, {slots, 8 * nt}};
  for (const Span& i : ins)
    for (const Span& o : outs) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(i.p), b = reinterpret_cast<uintptr_t>(o.p);
      if (a && i.bytes && a < b + o.bytes && b < a + i.bytes)
        return set_error(M3_EINVAL, "an output overlaps fresh, cached, free_pages or free_at");
    }
  if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots) |
       reinterpret_cast<uintptr_t>(seqs)) & 15)
    return set_error(M3_EINVAL, "positions, slots and seqs have to be 16-byte aligned");
  MapArgs a{fresh, cached, free_pages, free_at, table, cu, positions, seqs, lens, taken, slots,
            ld_table, n_req, n_free, max_pages, shift, n_pages, start, n_tokens};
  const long long by_tok = (n_tokens + 4ll * kMapThreads - 1) / (4ll * kMapThreads);
  const long long by_req = (n_req + 63) / 64;  // four requests' columns per warp
  long long grid = by_tok > by_req ? by_tok : by_req;
  const int nsm = sm_count();
  if (grid > 2 * nsm) grid = 2 * nsm;
  if (grid < 1) grid = 1;
  const size_t smem = sizeof(int) * (2 * (size_t)n_req + 1);
  if (smem > 40 * 1024)
    OPS_CK(cudaFuncSetAttribute(kv_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(int) * (2 * (size_t)kMapMaxReq + 1))));
  kv_map_kernel<<<(unsigned)grid, kMapThreads, smem, static_cast<cudaStream_t>(cuda_stream)>>>(a);
  OPS_CK(cudaGetLastError());
  return M3_OK;
}

extern "C" int m3_kv_store(int dtype, int n_tokens, int Hkv, int D, const void* k, int64_t k_token,
                           int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                           const int64_t* slots, void* pool, int n_pages, int page,
                           void* cuda_stream) {
  if (dtype != M3_KV_BF16 && dtype != M3_KV_F16) return set_error(M3_EINVAL, "dtype");
  if (n_tokens < 0 || n_pages < 0 || Hkv < 1 || Hkv > 1024)
    return set_error(M3_EINVAL, "n_tokens, n_pages or Hkv");
  if (D < 8 || D > 1024 || D % 8) return set_error(M3_EINVAL, "D: a multiple of 8, up to 1024");
  const int shift = page_shift(page);
  if (shift < 0) return set_error(M3_EINVAL, "page: a power of two, 16..1024");
  if (n_tokens == 0 || n_pages == 0) return M3_OK;
  if (!k || !v || !slots || !pool) return set_error(M3_EINVAL, "null argument");
  if (reinterpret_cast<uintptr_t>(pool) & 15)
    return set_error(M3_EINVAL, "the pool has to be 16-byte aligned");
  StoreArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_token, k_head,
              v_token, v_head, slots, static_cast<uint4*>(pool), (long long)n_pages << shift,
              n_tokens, Hkv, D / 8, shift};
  const bool vec = !((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) &&
                   !((k_token | k_head | v_token | v_head) & 7);
  const int ncol = 2 * Hkv * a.pieces, width = ncol < kStoreThreads ? ncol : kStoreThreads;
  const long long groups = kStoreThreads / width;
  long long grid = (n_tokens + groups - 1) / groups;
  const long long most = 8ll * sm_count();
  if (grid > most) grid = most;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (vec) kv_store_kernel<true><<<(unsigned)grid, kStoreThreads, 0, st>>>(a);
  else kv_store_kernel<false><<<(unsigned)grid, kStoreThreads, 0, st>>>(a);
  OPS_CK(cudaGetLastError());
  return M3_OK;
}

extern "C" int m3_logit_rules(int dtype, int n_rows, int vocab, const void* logits,
                              int64_t ld_logits, void* out, int64_t ld_out, const int32_t* history,
                              int n_history, int64_t ld_history, const int32_t* hist_len,
                              const float* repetition, const float* frequency,
                              const float* presence, const int32_t* bias_ids, const float* bias,
                              int n_bias, const uint32_t* mask, int n_masks,
                              const int32_t* mask_row, void* cuda_stream) {
  if (dtype != M3_LOGITS_F32 && dtype != M3_LOGITS_BF16 && dtype != M3_LOGITS_F16)
    return set_error(M3_EINVAL, "dtype");
  if (n_rows < 0 || vocab < 1 || vocab > (1 << 30)) return set_error(M3_EINVAL, "n_rows or vocab");
  if (n_history < 0 || n_history > kRuleMaxHistory || n_bias < 0 || n_bias > kRuleMaxBias ||
      n_masks < 0)
    return set_error(M3_EINVAL, "n_history (up to 2^24), n_bias (up to 4096) or n_masks");
  if (n_rows == 0) return M3_OK;
  if (!logits || !out) return set_error(M3_EINVAL, "null argument");
  if (n_bias && (!bias_ids || !bias)) return set_error(M3_EINVAL, "null bias_ids or bias");
  if (n_history && !history) return set_error(M3_EINVAL, "null history");
  if (mask && n_masks < 1) return set_error(M3_EINVAL, "a mask without n_masks");
  if (mask && !mask_row && n_masks != 1 && n_masks != n_rows)
    return set_error(M3_EINVAL, "without mask_row, n_masks is 1 or n_rows");
  if (n_rows > 1 && (ld_logits < vocab || ld_out < vocab || (n_history && ld_history < n_history)))
    return set_error(M3_EINVAL, "rows overlap");
  const int es = dtype == M3_LOGITS_F32 ? 4 : 2;
  const uintptr_t i0 = reinterpret_cast<uintptr_t>(logits), o0 = reinterpret_cast<uintptr_t>(out);
  if ((i0 | o0) & (es - 1)) return set_error(M3_EINVAL, "logits or out not aligned to their type");
  const uintptr_t ni = ((uintptr_t)(n_rows - 1) * ld_logits + vocab) * es;
  const uintptr_t no = ((uintptr_t)(n_rows - 1) * ld_out + vocab) * es;
  const bool same = i0 == o0 && (n_rows == 1 || ld_logits == ld_out);
  // rows of one stride may lie side by side, in columns of one buffer
  const uintptr_t ld = (uintptr_t)ld_logits * es, row = (uintptr_t)vocab * es;
  const uintptr_t apart = ld ? (o0 > i0 ? (o0 - i0) % ld : (ld - (i0 - o0) % ld) % ld) : 0;
  const bool beside = n_rows > 1 && ld_logits == ld_out && apart >= row && apart + row <= ld;
  if (!same && !beside && i0 < o0 + no && o0 < i0 + ni)
    return set_error(M3_EINVAL, "out overlaps logits without being logits");
  RuleArgs a{};
  a.in = logits;
  a.out = out;
  a.ld_in = ld_logits;
  a.ld_out = ld_out;
  a.history = n_history ? history : nullptr;
  a.ld_history = ld_history;
  a.hist_len = hist_len;
  a.rep = repetition;
  a.freq = frequency;
  a.pres = presence;
  a.bias_ids = bias_ids;
  a.bias = bias;
  a.mask = mask;
  a.mask_row = mask_row;
  a.vocab = vocab;
  a.n_history = n_history;
  a.n_bias = n_bias;
  a.n_masks = n_masks;
  a.words = (vocab + 31) / 32;
  // a run: the longest that still gives every SM a CTA, 1024 logits at least
  a.run = kRuleRun;
  while (a.run > 1024 && (((long long)vocab + 7 + a.run - 1) / a.run) * n_rows < sm_count())
    a.run >>= 1;
  a.runs = (int)(((long long)vocab + 7 + a.run - 1) / a.run);
  if ((long long)a.runs * n_rows > INT_MAX) return set_error(M3_EINVAL, "too many rows");
  if (same && !mask && !a.history && !n_bias) return M3_OK;
  // two launches from twelve runs of the longest per SM on, and where penalties or
  // biases alone touch logits in place
  if ((a.history || n_bias) &&
      ((same && !mask) || (long long)a.runs * n_rows >= 12ll * sm_count() * (kRuleRun / a.run)))
    a.parts = 1;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == M3_LOGITS_F32) OPS_CK(launch_rules<float>(a, n_rows, st));
  else if (dtype == M3_LOGITS_BF16) OPS_CK(launch_rules<__nv_bfloat16>(a, n_rows, st));
  else OPS_CK(launch_rules<__half>(a, n_rows, st));
  return M3_OK;
}
