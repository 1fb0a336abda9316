// kv_evict.cu -- eviction from the paged cache by accumulated attention
// weight.
//
// A sequence of L tokens keeps n = min(L, keep[b]) of them: its last
// `recent`, its first `sink`, and of the rest those with the largest weight
// (equal weights: the lower position; NaN below every number).  The kept
// tokens keep their order and move together to positions 0 .. n-1: K and V
// rows and weights, in place or into other blocks (a sequence whose blocks
// are shared is compacted into blocks of its own).  Each kv head chooses for
// itself, or all heads of a sequence by their summed weights.  The pages
// describe only whole sequences leaving the cache (vLLM concept page,
// compassingai.com, preemption); keeping part of one is this library's.
//
// Two launches.  evict_select_kernel: one CTA per choice finds the weight
// of the last kept token by radix selection over order-preserving 32-bit
// keys, then writes the kept positions in ascending order.  The second
// launch moves the rows: evict_gather_kernel into other blocks, every row
// independent, or evict_compact_kernel in place.
#include <algorithm>
#include <utility>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

static __device__ ErrorWord g_err_evict = {0ull, 0ull};

struct EvictParams {
  uint8_t *k_cache, *v_cache;
  const int32_t *tables, *dst_tables;  // dst_tables == tables: in place
  const int32_t *seq_lens, *keep;
  const float *weights;  // [batch, num_kv_heads, weights_stride]
  float *dst_weights;    // [batch, num_kv_heads, dst_stride]
  int32_t *new_seq_lens;
  int32_t *kept;    // [batch, choices, max_keep]
  int2 *counts;     // [batch]: (n, L), n < 0 where the sequence is left alone
  long long weights_stride, dst_stride;
  int32_t batch, num_kv_heads, choices;  // choices: num_kv_heads, or 1
  int32_t num_blocks, max_blocks, dst_max_blocks, max_keep, sink, recent;
  int32_t row_bytes;  // of one head's row
  int32_t weights_in_place;
};

// A float's bits as an unsigned key of the same order: -0 equals +0, NaN is
// below -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The ranking weight of token t: the head's, or the heads' sum (in binary64,
// heads in order, rounded once).
__device__ __forceinline__ float rank_weight(const EvictParams &p, int b, int h, int t) {
  const float *w = p.weights + (size_t)b * p.num_kv_heads * p.weights_stride;
  if (p.choices > 1 || p.num_kv_heads == 1) return w[(size_t)h * p.weights_stride + t];
  double s = 0.0;
  for (int k = 0; k < p.num_kv_heads; ++k) s += (double)w[(size_t)k * p.weights_stride + t];
  return (float)s;
}

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int pick[2];  // digit, elements wanted within it
  __shared__ int warp_gt[kSelectWarps], warp_eq[kSelectWarps];
  grid_dependency_wait();
  allow_dependent_launch();
  const int h = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t *kept = p.kept + ((size_t)b * p.choices + h) * p.max_keep;

  const int L = __ldg(p.seq_lens + b), want = __ldg(p.keep + b);
  const int n = min(L, want);
  const bool bad = L < 0 || want < 0 || (long long)L > (long long)p.max_blocks * 16 ||
                   L > p.weights_stride || n > p.max_keep || n > p.dst_stride ||
                   (long long)n > (long long)p.dst_max_blocks * 16;
  if (h == 0 && tid == 0) {
    p.counts[b] = make_int2(bad ? -1 : n, L);
    if (bad) record_error(&g_err_evict, PKV_ERR_RANGE, b);
  }
  for (int i = (bad ? 0 : n) + tid; i < p.max_keep; i += kSelectThreads) kept[i] = -1;
  if (bad) return;
  const int recent = min(p.recent, n), sink = min(p.sink, n - recent);
  // the middle: tokens sink .. L - recent - 1, of which k are kept
  const int mid = L - recent - sink, k = n - recent - sink;
  for (int i = tid; i < sink; i += kSelectThreads) kept[i] = i;
  for (int i = tid; i < recent; i += kSelectThreads) kept[n - recent + i] = L - recent + i;
  if (!p.weights_in_place) {
    // positions given up start from 0 (in place: once their weights are read)
    const int end = (int)min((long long)L, p.dst_stride);
    for (int hh = p.choices > 1 ? h : 0; hh < (p.choices > 1 ? h + 1 : p.num_kv_heads); ++hh) {
      float *w = p.dst_weights + ((size_t)b * p.num_kv_heads + hh) * p.dst_stride;
      for (int t = n + tid; t < end; t += kSelectThreads) w[t] = 0.f;
    }
  }
  if (k == 0) return;
  if (k == mid) {
    for (int i = tid; i < mid; i += kSelectThreads) kept[sink + i] = sink + i;
    return;
  }

  // the k-th largest key, 8 bits at a time from the top
  uint32_t prefix = 0;
  int left = k;  // wanted among the keys that share the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < mid; i += kSelectThreads) {
      const uint32_t key = weight_key(rank_weight(p, b, h, sink + i));
      if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8 l .. 248 - 8 l: counts from the top
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = hist[255 - 8 * lane - j];
        sum += c[j];
      }
      int above = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, above, off);
        if (lane >= off) above += o;
      }
      above -= sum;  // elements with a higher digit than this lane's first
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (above < left && left <= above + c[j]) {
          pick[0] = 255 - 8 * lane - j;
          pick[1] = left - above;
        }
        above += c[j];
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)pick[0];
    left = pick[1];
    __syncthreads();
  }
  // kept: every key above `prefix`, and the first `left` keys equal to it.
  // A warp owns a contiguous piece of the middle: count, scan, write.
  const int piece = (mid + kSelectThreads - 1) / kSelectThreads * 32;
  const int p0 = min(mid, warp * piece), p1 = min(mid, p0 + piece);
  int gt = 0, eq = 0;
  for (int i0 = p0; i0 < p1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < p1 ? weight_key(rank_weight(p, b, h, sink + i)) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < p1 && key > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < p1 && key == prefix));
  }
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int w = 0; w < warp; ++w) {
    gt += warp_gt[w];
    eq += warp_eq[w];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = p0; i0 < p1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < p1 ? weight_key(rank_weight(p, b, h, sink + i)) : 0u;
    const uint32_t m_gt = __ballot_sync(0xffffffffu, i < p1 && key > prefix);
    const uint32_t m_eq = __ballot_sync(0xffffffffu, i < p1 && key == prefix);
    const int my_eq = eq + __popc(m_eq & below);
    if (i < p1 && (key > prefix || (key == prefix && my_eq < left)))
      kept[sink + gt + __popc(m_gt & below) + min(my_eq, left)] = sink + i;
    gt += __popc(m_gt);
    eq += __popc(m_eq);
  }
}

// Row index (head rows of the pool) of position t through a table row; -1
// and an error when the block lies outside the pool.
__device__ __forceinline__ long long row_of(const EvictParams &p, const int32_t *table, int width,
                                            int b, int h, int t) {
  const int32_t blk = __ldg(table + (size_t)b * width + (t >> 4));
  if (blk < 0 || blk >= p.num_blocks) {
    record_error(&g_err_evict, PKV_ERR_RANGE, (long long)b * width + (t >> 4));
    return -1;
  }
  return ((long long)blk * 16 + (t & 15)) * p.num_kv_heads + h;
}

// Into other blocks: a warp moves 32 tokens of one (sequence, kv head).
// Lane i looks up token i's rows; then RB / 16 lanes move a row, 16 bytes
// each, K and V of several rows in flight.
constexpr int kGatherThreads = 128;

template <int RB>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictParams p) {
  constexpr int LANES = RB / 16, ROWS = 32 / LANES, STEPS = 32 / ROWS;
  constexpr int BATCH = STEPS < 4 ? STEPS : 4;
  grid_dependency_wait();
  allow_dependent_launch();
  const int b = blockIdx.z, h = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int2 c = p.counts[b];
  const int n = c.x;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.new_seq_lens[b] = n < 0 ? c.y : n;
  const int i0 = (blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5)) * 32;
  if (i0 >= n) return;
  const int i = i0 + lane;
  long long src = -1, dst = -1;
  if (i < n) {
    const int t =
        p.kept[((size_t)b * p.choices + (p.choices > 1 ? h : 0)) * p.max_keep + i];
    src = row_of(p, p.tables, p.max_blocks, b, h, t);
    dst = row_of(p, p.dst_tables, p.dst_max_blocks, b, h, i);
    if (src < 0 || dst < 0) src = dst = -1;
    if (!p.weights_in_place) {
      const size_t bh = (size_t)b * p.num_kv_heads + h;
      p.dst_weights[bh * p.dst_stride + i] = p.weights[bh * p.weights_stride + t];
    }
  }
  const int sub = lane / LANES, u = lane % LANES;
  const uint4 *ks = reinterpret_cast<const uint4 *>(p.k_cache);
  const uint4 *vs = reinterpret_cast<const uint4 *>(p.v_cache);
  uint4 *kd = reinterpret_cast<uint4 *>(p.k_cache), *vd = reinterpret_cast<uint4 *>(p.v_cache);
#pragma unroll
  for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
    uint4 kr[BATCH], vr[BATCH];
    long long to[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int r = (s0 + k) * ROWS + sub;
      const long long from = __shfl_sync(0xffffffffu, src, r);
      to[k] = __shfl_sync(0xffffffffu, dst, r);
      if (from >= 0) {
        kr[k] = ks[from * LANES + u];
        vr[k] = vs[from * LANES + u];
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (to[k] >= 0) {
        kd[to[k] * LANES + u] = kr[k];
        vd[to[k] * LANES + u] = vr[k];
      }
  }
}

// In place: token kept[i] moves to position i <= kept[i].  One CTA takes one
// plane (K, V or the weights) of one (sequence, kv head) and walks it in
// chunks in ascending order: a chunk is read whole before it is written, and
// every later chunk's sources lie at or above its own positions, past all
// positions written so far.
constexpr int kCompactThreads = 256;
constexpr int kCompactTokens = 128;

template <int RB>
__global__ void __launch_bounds__(kCompactThreads) evict_compact_kernel(const EvictParams p) {
  constexpr int LANES = RB / 16;
  constexpr int PER = kCompactTokens * LANES / kCompactThreads;  // vectors of a thread
  __shared__ long long from_s[2][kCompactTokens], to_s[2][kCompactTokens];
  grid_dependency_wait();
  allow_dependent_launch();
  const int b = blockIdx.z, h = blockIdx.y, plane = blockIdx.x;
  const int tid = threadIdx.x;
  const int2 c = p.counts[b];
  const int n = c.x, L = c.y;
  if (plane == 0 && h == 0 && tid == 0) p.new_seq_lens[b] = n < 0 ? L : n;
  const bool moves = p.dst_tables == p.tables;  // K and V in place
  if (n < 0) return;                            // left alone
  const int32_t *kept = p.kept + ((size_t)b * p.choices + (p.choices > 1 ? h : 0)) * p.max_keep;
  if (plane == 2) {
    const size_t bh = (size_t)b * p.num_kv_heads + h;
    float *w = p.dst_weights + bh * p.dst_stride;
    if (!p.weights_in_place) {  // (into other blocks: moved with the rows)
      const float *from = p.weights + bh * p.weights_stride;
      if (moves)
        for (int i = tid; i < n; i += kCompactThreads) w[i] = from[kept[i]];
      return;
    }
    if (n == L) return;  // nothing given up
    for (int i0 = 0; i0 < n; i0 += kCompactThreads) {
      const int i = i0 + tid;
      const float x = i < n ? w[kept[i]] : 0.f;
      __syncthreads();
      if (i < n) w[i] = x;
    }
    __syncthreads();
    for (int t = n + tid; t < L; t += kCompactThreads) w[t] = 0.f;
    return;
  }
  if (!moves || n == L) return;
  uint4 *pool = reinterpret_cast<uint4 *>(plane == 0 ? p.k_cache : p.v_cache);
  for (int i0 = 0; i0 < n; i0 += kCompactTokens) {
    const int buf = (i0 / kCompactTokens) & 1;
    if (tid < kCompactTokens) {
      long long from = -1, to = -1;
      if (i0 + tid < n) {
        const int t = kept[i0 + tid];
        if (t != i0 + tid) {  // (a token that stays needs no copy)
          from = row_of(p, p.tables, p.max_blocks, b, h, t);
          to = row_of(p, p.tables, p.max_blocks, b, h, i0 + tid);
          if (from < 0 || to < 0) from = to = -1;
        }
      }
      from_s[buf][tid] = from;
      to_s[buf][tid] = to;
    }
    __syncthreads();
    uint4 x[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int idx = k * kCompactThreads + tid;
      const long long from = from_s[buf][idx / LANES];
      if (from >= 0) x[k] = pool[from * LANES + idx % LANES];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int idx = k * kCompactThreads + tid;
      const long long to = to_s[buf][idx / LANES];
      if (to >= 0) pool[to * LANES + idx % LANES] = x[k];
    }
  }
}

namespace {

size_t counts_bytes(int64_t batch) { return ((size_t)batch * sizeof(int2) + 255) / 256 * 256; }

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s,
                       Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int RB>
cudaError_t launch_move(const EvictParams &p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool in_place = p.dst_tables == p.tables;
  const int per = kGatherThreads;  // tokens of a CTA
  if (!in_place)
    e = launch_pdl(evict_gather_kernel<RB>,
                   dim3(std::max(1, (p.max_keep + per - 1) / per), p.num_kv_heads, p.batch),
                   dim3(kGatherThreads), s, p);
  if (e == cudaSuccess && (in_place || p.weights_in_place))
    e = launch_pdl(evict_compact_kernel<RB>, dim3(3, p.num_kv_heads, p.batch),
                   dim3(kCompactThreads), s, p);
  return e;
}

bool overlap(const void *a, size_t a_len, const void *b, size_t b_len) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_len && y < x + a_len;
}

}  // namespace

const void *error_word_evict() { return &g_err_evict; }

}  // namespace pkv

using namespace pkv;

extern "C" size_t paged_kv_evict_workspace_bytes(int32_t batch, int32_t num_kv_heads,
                                                 int64_t weights_stride, int32_t max_keep) {
  if (batch <= 0 || num_kv_heads <= 0 || weights_stride < 0 || max_keep < 0) return 0;
  return counts_bytes(batch) +
         ((size_t)batch * num_kv_heads * max_keep * sizeof(int32_t) + 255) / 256 * 256;
}

extern "C" pkv_status paged_kv_evict(const pkv_cache *cache, const int32_t *block_tables,
                                     int32_t max_blocks, const int32_t *seq_lens,
                                     float *weights, int64_t weights_stride, const int32_t *keep,
                                     int32_t batch, int32_t max_keep, int32_t sink, int32_t recent,
                                     int per_head, const int32_t *dst_tables,
                                     int32_t dst_max_blocks, float *dst_weights,
                                     int64_t dst_weights_stride, int32_t *new_seq_lens,
                                     int32_t *kept, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  pkv_status st = validate_cache(cache);
  if (st != PKV_OK) return st;
  if (batch < 0 || max_blocks <= 0 || max_keep < 0 || sink < 0 || recent < 0 ||
      weights_stride < 0 || (dst_tables && dst_max_blocks <= 0) ||
      (dst_weights && dst_weights_stride < 0))
    return PKV_ERR_ARG;
  if (batch == 0) return PKV_OK;
  if (!block_tables || !seq_lens || !weights || !keep || !new_seq_lens) return PKV_ERR_ARG;
  if (batch > 65535 || cache->num_kv_heads > 65535 || weights_stride > INT32_MAX ||
      (dst_weights && dst_weights_stride > INT32_MAX) || max_keep > INT32_MAX - 1024)
    return PKV_ERR_ARG;
  const size_t rows = (size_t)batch * cache->num_kv_heads;
  // other weights must not lie over the ones still to be read
  if (dst_weights && overlap(weights, rows * weights_stride * 4, dst_weights,
                             rows * dst_weights_stride * 4))
    return PKV_ERR_ARG;
  // (new_seq_lens may be seq_lens: it is written after the last read)
  if (new_seq_lens != seq_lens && overlap(new_seq_lens, 4 * (size_t)batch, seq_lens,
                                          4 * (size_t)batch))
    return PKV_ERR_ARG;
  if (overlap(new_seq_lens, 4 * (size_t)batch, keep, 4 * (size_t)batch)) return PKV_ERR_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      workspace_bytes < paged_kv_evict_workspace_bytes(batch, cache->num_kv_heads, weights_stride,
                                                       max_keep))
    return PKV_ERR_WORKSPACE;
  EvictParams p = {};
  p.k_cache = static_cast<uint8_t *>(cache->key_cache);
  p.v_cache = static_cast<uint8_t *>(cache->value_cache);
  p.tables = block_tables;
  p.dst_tables = dst_tables ? dst_tables : block_tables;
  p.seq_lens = seq_lens;
  p.keep = keep;
  p.weights = weights;
  p.dst_weights = dst_weights ? dst_weights : weights;
  p.weights_in_place = dst_weights == nullptr;
  p.new_seq_lens = new_seq_lens;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.counts = reinterpret_cast<int2 *>(ws);
  p.kept = kept ? kept : reinterpret_cast<int32_t *>(ws + counts_bytes(batch));
  p.weights_stride = weights_stride;
  p.dst_stride = dst_weights ? dst_weights_stride : weights_stride;
  p.batch = batch;
  p.num_kv_heads = cache->num_kv_heads;
  p.choices = per_head ? cache->num_kv_heads : 1;
  p.num_blocks = cache->num_blocks;
  p.max_blocks = max_blocks;
  p.dst_max_blocks = dst_tables ? dst_max_blocks : max_blocks;
  p.max_keep = max_keep;
  p.sink = sink;
  p.recent = recent;
  p.row_bytes = cache->head_dim * (cache->dtype == PKV_FP8_E4M3 ? 1 : 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_pdl(evict_select_kernel, dim3(p.choices, batch), dim3(kSelectThreads), s, p) !=
      cudaSuccess)
    return PKV_ERR_CUDA;
  const cudaError_t e = p.row_bytes == 256   ? launch_move<256>(p, s)
                        : p.row_bytes == 128 ? launch_move<128>(p, s)
                                             : launch_move<64>(p, s);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
