// Block tables and slot maps of a step, from the requests' lengths
// (mla_extend_tables): keeps the block_table and cache_seqlens that the decode
// calls take ("Qu'est-ce que FlashMLA ?", section "Exécuter le décodage MLA")
// up to date on the device.
//
//   need[b]  = ceil((ctx + new) / 64) - ceil(ctx / 64)       pages to add
//   place[b] = sum of need before b                          in the free list
//   start[b] = sum of new before b                           on the token axis
//   slot(t)  = page(b, pos / 64) * 64 + pos % 64,  pos = ctx[b] + t - start[b]
//
// Both sums depend on every request before b, everything else only on b. A
// step moves kilobytes (16 bytes a request, 8 a token): it is bound by the
// launch and by round trips, so there is one launch, and no block waits for
// another. Every block forms the sums itself, with the totals carried from
// pass to pass, and writes its share of the requests and of the tokens.
// Repeating the sums costs a block two loads and a scan per pass; a second
// launch or a grid-wide wait would cost more. Nothing that a
// block reads is written by another (the caller's buffers must not overlap,
// and of a table row only entries before the new ones are read).
#include <cuda_runtime.h>

#include "mla_kernels.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kItems = 4;            // requests of a pass per thread
constexpr int kTokensPerBlock = 1024;
constexpr int kShortRow = 4;         // new pages a thread writes itself; longer rows take a warp

// Two block sizes: 256 threads cover 1024 requests a pass; above that 1024
// threads cover 4096 (4096 requests: 6.6 us as one pass of the large block,
// 12.9 us as four of the small one; 128 requests: 5.0 us against 3.7 us).
constexpr int kSmall = 256, kLarge = 1024;

struct TableParams {
  const int32_t *ctx, *add, *free_pages, *free_range;
  int32_t *block_table, *seqlens, *token_start, *slots, *positions, *free_next;
  uint32_t* status;
  int batch, num_free, num_pages, stride, max_tokens;
};

struct Sums {
  long long tok, pages;
};
// Exclusive sums over the block, and the totals. Every warp scans the warps'
// totals itself, which saves a barrier.
template <int THREADS>
__device__ __forceinline__ Sums scan_block(Sums v, Sums& total, Sums* part) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, s.tok, o), y = __shfl_up_sync(0xffffffffu, s.pages, o);
    if (lane >= o) s.tok += x, s.pages += y;
  }
  __syncthreads();  // the last use of part is over
  if (lane == 31) part[warp] = s;
  __syncthreads();
  Sums w = {0, 0};
  if (lane < kWarps) w = part[lane];
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, w.tok, o), y = __shfl_up_sync(0xffffffffu, w.pages, o);
    if (lane >= o) w.tok += x, w.pages += y;
  }
  total.tok = __shfl_sync(0xffffffffu, w.tok, kWarps - 1);
  total.pages = __shfl_sync(0xffffffffu, w.pages, kWarps - 1);
  const long long bt = __shfl_sync(0xffffffffu, w.tok, max(warp - 1, 0)), bp = __shfl_sync(0xffffffffu, w.pages, max(warp - 1, 0));
  s.tok += (warp > 0 ? bt : 0) - v.tok;
  s.pages += (warp > 0 ? bp : 0) - v.pages;
  return s;
}

__device__ __forceinline__ int clamp_int(long long v) { return v < 0x7fffffffLL ? (int)v : 0x7fffffff; }
__device__ __forceinline__ int pages_of(long long tokens) { return (int)((tokens + kPage - 1) / kPage); }

template <int THREADS>
__global__ void __launch_bounds__(THREADS) extend_tables_kernel(const TableParams p) {
  constexpr int kPass = THREADS * kItems;
  extern __shared__ int s_lists[];
  int* s_start = s_lists;              // [kPass + 1]: first token of each request of the pass, then the pass's end
  int* s_ctx = s_start + kPass + 4;    // [kPass]: -1: refused
  int* s_base = s_ctx + kPass;         // [kPass]: free-list place of logical page j: base + j
  __shared__ Sums part[THREADS / 32];
  __shared__ int s_taken, s_long;
  griddep_wait();
  const int tid = threadIdx.x;
  uint32_t bits = 0;
  const int first = p.free_range[0], last = p.free_range[1];
  const int t0 = blockIdx.x * kTokensPerBlock, t1 = min(p.max_tokens, t0 + kTokensPerBlock);
  int avail = 0;
  auto fresh_page = [&](int place) {  // page id at a place of the free list; -1 if it is none
    const int pg = p.free_pages[place];
    if (pg >= 0 && pg < p.num_pages) return pg;
    bits |= MLA_DEVICE_STATUS_BOUNDS;
    return -1;
  };
  if (tid == 0) s_taken = 0, s_long = 0;
  Sums carry = {0, 0};
  for (int b0 = 0; b0 < p.batch; b0 += kPass) {
    const int n = min(kPass, p.batch - b0), i0 = tid * kItems;
    int ctx[kItems], add[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const bool in = i0 + k < n;
      ctx[k] = in ? p.ctx[b0 + i0 + k] : 0;
      add[k] = in ? p.add[b0 + i0 + k] : 0;
    }
    if (b0 == 0) {  // looked at only now, so that its load and the first lengths' are one round trip
      const bool range_ok = first >= 0 && first <= last && last <= p.num_free;
      avail = range_ok ? last - first : 0;
      if (!range_ok) bits |= MLA_DEVICE_STATUS_BOUNDS;
    }
    // a request is in order if its lengths are, its row holds them and its tokens end in time
    uint32_t ok = 0;
    int need[kItems];
    Sums mine = {0, 0}, total;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const long long len = (long long)ctx[k] + add[k];
      need[k] = 0;
      if (ctx[k] >= 0 && add[k] >= 0 && len <= (long long)p.stride * kPage) {
        ok |= 1u << k;
        need[k] = pages_of(len) - pages_of(ctx[k]);
      }
      mine.tok += max(add[k], 0);
      mine.pages += need[k];
    }
    Sums at = scan_block<THREADS>(mine, total, part);
    if (carry.tok + total.tok > p.max_tokens) {  // some tokens end past the axis: their requests need no pages
      long long tok = carry.tok + at.tok;
      mine.pages = 0;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        tok += max(add[k], 0);
        if (tok > p.max_tokens) {
          ok &= ~(1u << k);
          need[k] = 0;
        }
        mine.pages += need[k];
      }
      at = scan_block<THREADS>(mine, total, part);
    }
    long long tok = carry.tok + at.tok, pages = carry.pages + at.pages;
    carry.tok += total.tok;
    carry.pages += total.pages;
    if (tid == 0) s_start[n] = clamp_int(carry.tok);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (i0 + k < n) {
        bool served = (ok >> k) & 1u;
        if (!served) bits |= MLA_DEVICE_STATUS_BOUNDS;
        // without enough pages; then the later ones that need some have none either, as the sum only grows
        if (need[k] > 0 && pages + need[k] > avail) {
          served = false;
          bits |= MLA_DEVICE_STATUS_NO_PAGES;
        }
        s_start[i0 + k] = clamp_int(tok);
        s_ctx[i0 + k] = served ? ctx[k] : -1;
        s_base[i0 + k] = served ? first + (int)pages - pages_of(ctx[k]) : 0;
        if (served && need[k] > 0) atomicMax(&s_taken, (int)pages + need[k]);
        if (served && need[k] > kShortRow) s_long = 1;
      }
      tok += max(add[k], 0);
      pages += need[k];
    }
    __syncthreads();
    // this block's requests: every gridDim.x-th group of THREADS; long rows by warps
    for (int i = blockIdx.x * THREADS + tid; i < n; i += gridDim.x * THREADS) {
      const int b = b0 + i, c = s_ctx[i], a = s_start[i + 1] - s_start[i];
      p.token_start[b] = s_start[i];
      p.seqlens[b] = c >= 0 ? c + a : max(p.ctx[b], 0);
      if (c < 0) continue;
      const int h = pages_of(c), e = pages_of((long long)c + a);
      if (e - h <= kShortRow)
        for (int j = h; j < e; ++j) p.block_table[(size_t)b * p.stride + j] = fresh_page(s_base[i] + j);
    }
    if (s_long)
      for (int i = blockIdx.x * (THREADS / 32) + (tid >> 5); i < n; i += gridDim.x * (THREADS / 32)) {
        const int c = s_ctx[i], a = s_start[i + 1] - s_start[i];
        if (c < 0) continue;
        const int h = pages_of(c), e = pages_of((long long)c + a);
        if (e - h > kShortRow)
          for (int j = h + (tid & 31); j < e; j += 32)
            p.block_table[(size_t)(b0 + i) * p.stride + j] = fresh_page(s_base[i] + j);
      }
    // this block's tokens of the pass
    for (int t = max(t0, s_start[0]) + tid; t < min(t1, s_start[n]); t += THREADS) {
      int lo = 0, hi = n - 1;  // the last request that starts at or before t is the one that has it
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (s_start[m] <= t) lo = m;
        else hi = m - 1;
      }
      const int c = s_ctx[lo];
      int pos = -1, slot = -1;
      if (c >= 0) {
        pos = c + (t - s_start[lo]);  // c + t may pass 2^31
        const int j = pos / kPage;
        int pg;
        if ((long long)j * kPage >= c) {
          pg = fresh_page(s_base[lo] + j);
        } else {  // the request's last page so far
          pg = p.block_table[(size_t)(b0 + lo) * p.stride + j];
          if (pg < 0 || pg >= p.num_pages) {
            bits |= MLA_DEVICE_STATUS_BOUNDS;
            pg = -1;
          }
        }
        if (pg >= 0) slot = pg * kPage + pos % kPage;
      }
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
    __syncthreads();  // before the next pass rewrites the lists
  }
  for (long long t = max((long long)t0, carry.tok) + tid; t < t1; t += THREADS) {  // behind the last token
    p.slots[t] = -1;
    p.positions[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.token_start[p.batch] = clamp_int(carry.tok);
    p.free_next[0] = first + s_taken;
  }
  if (bits != 0 && p.status != nullptr) atomicOr(p.status, bits);
}

template <int THREADS>
cudaError_t launch_tables(const TableParams& p, cudaStream_t stream) {
  constexpr int smem = (3 * THREADS * kItems + 4) * (int)sizeof(int);
  auto kern = extend_tables_kernel<THREADS>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3((p.max_tokens - 1) / kTokensPerBlock + 1), dim3(THREADS), smem, stream, p);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_extend_tables(const int32_t* context_lens, const int32_t* new_lens, int batch,
                                          const int32_t* free_pages, int num_free, const int32_t* free_range,
                                          int num_pages, int32_t* block_table, int block_table_stride,
                                          int32_t* seqlens, int32_t* token_start, int32_t* slots, int32_t* positions,
                                          int max_tokens, int32_t* free_next, uint32_t* status, mla_stream_t stream) {
  if (batch <= 0 || num_free < 0 || num_pages <= 0 || block_table_stride <= 0 || max_tokens <= 0)
    return MLA_ERR_INVALID_ARG;
  if (!free_pages && num_free > 0) return MLA_ERR_INVALID_ARG;
  const struct { const void* p; size_t n; } in[] = {{context_lens, (size_t)batch * 4}, {new_lens, (size_t)batch * 4},
                                                    {free_range, 8}, {free_pages, (size_t)num_free * 4}};
  const struct { const void* p; size_t n; } out[] = {
      {block_table, (size_t)batch * block_table_stride * 4}, {seqlens, (size_t)batch * 4},
      {token_start, ((size_t)batch + 1) * 4}, {slots, (size_t)max_tokens * 4}, {positions, (size_t)max_tokens * 4},
      {free_next, 4}, {status, status ? sizeof(*status) : 0}};
  for (int i = 0; i < 4; ++i)
    if ((!in[i].p && i < 3) || !aligned4(in[i].p)) return MLA_ERR_INVALID_ARG;
  for (int i = 0; i < 7; ++i) {
    if ((!out[i].p && i < 6) || !aligned4(out[i].p)) return MLA_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return MLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return MLA_ERR_INVALID_ARG;
  }
  if ((long long)num_pages * kPage > 0x7fffffffLL || (long long)block_table_stride * kPage > 0x7fffffffLL ||
      batch > (1 << 30) || max_tokens > (1 << 30))
    return MLA_ERR_UNSUPPORTED;
  TableParams p{context_lens, new_lens, free_pages, free_range, block_table, seqlens, token_start, slots, positions,
                free_next, status, batch, num_free, num_pages, block_table_stride, max_tokens};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = batch <= kSmall * kItems ? launch_tables<kSmall>(p, st) : launch_tables<kLarge>(p, st);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
