// MLA decode over the 4-bit cache (MLA_KV_FP4_E2M1 records), units of at most
// 64 query rows: one CTA per scheduler part, paged or token-sparse.
//
// Same computation and TMEM layout as the row-group kernel of the bf16 cache
// (mla_decode.cu): per tile of 128 tokens
//   S    = Q K^T     tcgen05 M=64 rows x N=128 tokens x K=576 (f16, RoPE bf16)
//   softmax          one thread per query row, online, O rescaled lazily
//   O^T += V^T P^T   tcgen05 M=128 value dims (4 chunks) x N=rows x K=128
// The keys reach the tensor core through one ring of 32 KB entries that is
// filled from the records (mla_fp4.cuh), in the order in which
// the one MMA issuer consumes it: S(0), S(1), O(0), S(2), O(1), ...
//
// Warp roles (640 threads):
//   0 Q via TMA   1 MMA issuer (+ TMEM alloc)   2 cache rows   3 RoPE slices
//   4-7 softmax + epilogue (row r = 16*(warp-4) + lane, lanes 0-15)
//   8-11 raw copies   12-19 converters (and Q into form)
// Every wait is bounded; on a timeout the CTA records
// MLA_DEVICE_STATUS_TIMEOUT, stops issuing work, waits (bounded) for its own
// copies and MMAs and exits normally.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mla_fp4.cuh"

namespace mla {
namespace {

using fp4::kN;
constexpr int kQBytes = 9 * 8192;      // 64 rows x 576 dims
constexpr int kTmemCols = 512;
constexpr int kTmemS = 256;            // S buffers at columns 256 and 384
constexpr float kRescaleLog2 = 8.0f;   // rescale O only when the max grows by > 2^8

struct Ctrl {
  uint64_t q_raw, q_full, q_empty;      // q_raw: as loaded; q_full: converter warps have it in form
  uint64_t full[kN], empty[kN];
  uint64_t rope_free;                   // entry 1 of a K phase is consumed
  uint64_t s_full[2];
  uint64_t p_full, o_done, o_free, drain;
  uint64_t grp_sm;  // bounded barrier of the 128 softmax threads
  float q_back[2][64];                 // [piece parity][row]: what undoes the query's scaling
  uint32_t tmem_base;
  int abort_flag;
  int rescale_flag[2];
  float alpha[64];
  float inv_l[64];
};
static_assert(sizeof(Ctrl) <= 1536, "control block");

template <int NR>
struct Smem {
  static constexpr int q = 0;
  static constexpr int ring = q + kQBytes;
  static constexpr int raw = ring + kN * fp4::kSlot;
  static constexpr int pt = (raw + fp4::kRaw * fp4::kRawBytes + 1023) / 1024 * 1024;  // swizzled
  static constexpr int pt_bytes = NR * 256;  // [NR rows][128 tokens] f16
  static constexpr int ctrl = pt + pt_bytes;
  static constexpr int rows = ctrl + 1536;
  static constexpr int total = rows + (int)sizeof(fp4::RowTable);
};
static_assert(Smem<64>::total + 1024 <= 232448, "shared memory budget");

__device__ __forceinline__ bool timed_wait(Ctrl* c, uint64_t* bar, uint32_t parity, const DecodeParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*(volatile int*)&c->abort_flag) return false;
  if (mbar_wait(bar, parity, p.timeout_ns)) return true;
  atomicOr(p.status, (uint32_t)MLA_DEVICE_STATUS_TIMEOUT);
  *(volatile int*)&c->abort_flag = 1;
  return false;
}

// For all lanes of a warp that goes on to collective instructions: either all of
// them go on or, if the limit ran out for one, none.
__device__ __forceinline__ bool timed_wait_all(Ctrl* c, uint64_t* bar, uint32_t parity, const DecodeParams& p) {
  return __all_sync(0xffffffffu, timed_wait(c, bar, parity, p)) != 0;
}

// Barrier among the softmax threads, built on an mbarrier so the wait is
// bounded (a named barrier would hang if a member gave up).
__device__ __forceinline__ bool group_sync(Ctrl* c, uint64_t* bar, uint32_t& phase, const DecodeParams& p) {
  mbar_arrive(bar);
  const bool ok = timed_wait_all(c, bar, phase & 1, p);
  ++phase;
  return ok;
}

__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// O^T (value dims 128 m + the thread's on TMEM lanes, rows on columns) times
// the rows' factors -> the rows below `rows`, kDv apart, at dst + 128 m.
template <int NR, typename T>
__device__ __forceinline__ void store_rows(T* dst, uint32_t taddr, const float* inv_l, int rows) {
#pragma unroll 1
  for (int c16 = 0; c16 < NR / 16; ++c16, dst += 16 * kDv) {
    const int n = rows - 16 * c16;
    if (n <= 0) break;
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = inv_l[16 * c16 + i];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t ov[16];
      tmem_ld16(taddr + 64 * m + 16 * c16, ov);
      tmem_ld_wait();
      if (n >= 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) put(dst + i * kDv + 128 * m, __uint_as_float(ov[i]) * f[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n) put(dst + i * kDv + 128 * m, __uint_as_float(ov[i]) * f[i]);
      }
    }
  }
}

template <int NR, bool SPARSE>
__global__ void __launch_bounds__(fp4::kThreads, 1)
    mla_decode_fp4_kernel(const __grid_constant__ CUtensorMap tm_q, const DecodeParams p) {
  using L = Smem<NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::q;
  uint8_t* sRing = smem + L::ring;
  uint8_t* sRaw = smem + L::raw;
  uint8_t* sP = smem + L::pt;
  Ctrl* c = reinterpret_cast<Ctrl*>(smem + L::ctrl);
  fp4::RowTable* rt = reinterpret_cast<fp4::RowTable*>(smem + L::rows);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: known to be uniform
  const int part = blockIdx.x, row0 = 0;
  const int rows_here = p.rows;  // at most 64

  if (threadIdx.x == 0) {
    mbar_init(&c->q_raw, 1);
    mbar_init(&c->q_full, fp4::kCvWarps);
    mbar_init(&c->q_empty, 1);
    mbar_init(&c->rope_free, 1);
    for (int i = 0; i < kN; ++i) { mbar_init(&c->full[i], 4); mbar_init(&c->empty[i], 1); }
    for (int i = 0; i < 2; ++i) mbar_init(&c->s_full[i], 1);
    for (int i = 0; i < fp4::kRowDepth; ++i) {
      mbar_init(&rt->full[i], 1);
      mbar_init(&rt->empty[i], fp4::kLdWarps + 1 + (SPARSE ? 4 : 0));
    }
    for (int i = 0; i < fp4::kRaw; ++i) {
      mbar_init(&rt->raw_full[i], 32 * fp4::kLdWarps);
      mbar_init(&rt->raw_empty[i], 4);
    }
    mbar_init(&c->p_full, 128);
    mbar_init(&c->o_done, 1);
    mbar_init(&c->o_free, 128);
    mbar_init(&c->drain, 1);
    mbar_init(&c->grp_sm, 128);
    c->abort_flag = 0;
    c->rescale_flag[0] = 0;
    c->rescale_flag[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_q);
  if (warp == 1) {
    tmem_alloc(&c->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;
  griddep_wait();  // the scheduler's output (and every input) is ready

  PieceIter it;
  it.init(p, part);
  Piece pc;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return timed_wait(c, bar, parity, p); };
  auto full = [&](int slot) { return &c->full[slot]; };
  auto arrive = [&](int slot, int) { mbar_arrive(&c->full[slot]); };

  if (warp == 0) {
    // ------------------------------------------------------------ Q
    if (lane == 0) {
      int pi = 0, q_issued = 0;
      while (it.next(pc)) {
        if (!timed_wait(c, &c->q_empty, (pi & 1) ^ 1, p)) break;
        mbar_arrive_expect_tx(&c->q_raw, kQBytes);
        for (int j = 0; j < 9; ++j) tma_load_2d(sQ + j * 8192, &tm_q, &c->q_raw, 64 * j, pc.unit * p.rows);
        ++q_issued;
        ++pi;
      }
      if (q_issued > 0) mbar_wait(&c->q_raw, (uint32_t)((q_issued - 1) & 1), p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 2) {
    fp4::row_warp<false, SPARSE>(p, it, rt, lane, 0, wait);
  } else if (warp == 3) {
    fp4::load_rope<false>(p, it, rt, sRing, &c->rope_free, lane, 0, wait, full, arrive);
  } else if (warp >= 8 && warp < 12) {
    fp4::load_raw<false>(p, it, rt, sRaw, warp - 8, lane, 0, wait);
  } else if (warp >= 12) {
    fp4::convert_ring<false>(it, rt, sRing, sRaw, c->empty, warp - 12, lane, wait, arrive, [&](int piece) {
      if (!fp4::wait_warp(&c->q_raw, piece & 1, wait)) return false;
      fp4::scale_query_rows(sQ, c->q_back[piece & 1], rows_here, warp - 12, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->q_full);
      return true;
    });
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: S(0), S(1), O(0), S(2), O(1), ...
    if (elect_one()) {
      const uint32_t idesc_s = idesc_f16(64, 128, false, false), idesc_r = idesc_bf16(64, 128, false, false);
      const uint32_t idesc_o = idesc_f16(128, NR, true, false);
      // descriptors: Q, K and P^T are K-major, V is MN-major (slices 16 KB apart)
      const uint32_t q_lo = sdesc_lo(smem_u32(sQ), 16), k_lo = sdesc_lo(smem_u32(sRing), 16);
      const uint32_t v_lo = sdesc_lo(smem_u32(sRing), fp4::kSlice), p_lo = sdesc_lo(smem_u32(sP), 16);
      constexpr uint32_t d_hi = sdesc_hi(1024);
      int gs = 0, go = 0, pi = 0;
      fp4::RingPos pos;
      bool stop = false;
      while (!stop && it.next(pc)) {
        if (!timed_wait(c, &c->q_full, pi & 1, p)) break;
        const int nsteps = fp4::steps_of<false>(pc);
        for (int h = 0; h <= 2 * nsteps && !stop; ++h) {
          if (!fp4::phase_exists(h, nsteps)) continue;
          const int g = fp4::phase_step(h);
          if (fp4::phase_is_k(h)) {
            // S buffer b was last read by the softmax of tile gs - 2, whose
            // P the O product of that tile (issued before) waited for
            const uint32_t d = tmem + kTmemS + 128 * (gs & 1);
            for (int e = 0; e < 5; ++e, pos.advance()) {  // four latent entries of two slices, then RoPE
              const int slot = pos.slot;
              if (!timed_wait(c, &c->full[slot], pos.parity, p)) { stop = true; break; }
              if (e == 4) fence_proxy_async_smem();  // RoPE comes by cp.async
              tc_fence_after();
              const uint32_t qa = q_lo + 2 * e * (8192 >> 4), kb = k_lo + slot * (fp4::kSlot >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                if (kk < 4 || e < 4)
                  mma_bf16_ss(d, sdesc_join(qa + (kk >> 2) * (8192 >> 4) + (kk & 3) * 2, d_hi),
                              sdesc_join(kb + (kk >> 2) * (fp4::kSlice >> 4) + (kk & 3) * 2, d_hi), e < 4 ? idesc_s : idesc_r,
                              (e | kk) != 0 ? 1u : 0u);
              mma_commit(&c->empty[slot]);
              if (e == 1) mma_commit(&c->rope_free);
            }
            if (stop) break;
            if (!(gs == 0 && (p.debug_flags & MLA_DEBUG_WITHHOLD_SCORES))) mma_commit(&c->s_full[gs & 1]);
            ++gs;
            if (g == nsteps - 1) mma_commit(&c->q_empty);  // Q is free once the last S completes
          } else {
            const bool first = g == 0;
            if (first && pi > 0 && !timed_wait(c, &c->o_free, (pi - 1) & 1, p)) { stop = true; break; }
            if (!timed_wait(c, &c->p_full, go & 1, p)) { stop = true; break; }
            for (int m = 0; m < 4; ++m, pos.advance()) {  // value dims 128 m ..
              const int slot = pos.slot;
              if (!timed_wait(c, &c->full[slot], pos.parity, p)) { stop = true; break; }
              tc_fence_after();
              const uint32_t va = v_lo + slot * (fp4::kSlot >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ss(tmem + 64 * m, sdesc_join(va + kk * (2048 >> 4), d_hi),
                            sdesc_join(p_lo + (kk >> 2) * (NR * 128 >> 4) + (kk & 3) * 2, d_hi), idesc_o,
                            (first && kk == 0) ? 0u : 1u);
              mma_commit(&c->empty[slot]);
            }
            if (stop) break;
            mma_commit(&c->o_done);
            ++go;
          }
        }
        ++pi;
      }
      mma_commit(&c->drain);  // every MMA this thread issued has completed before TMEM is released
      mbar_wait(&c->drain, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ softmax + epilogue
    const int q4 = warp - 4;
    const int r = 16 * q4 + lane;                        // query row of this CTA (lanes 0-15)
    const bool owner = lane < 16;
    const bool rvalid = owner && r < rows_here;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    uint32_t gph = 0;
    int gt = 0, pi = 0;
    bool stop = false;
    while (!stop && it.next(pc)) {
      const int req = unit_req(p, pc.unit);
      const int grow = row0 + r;                          // row within the unit
      // lanes without a row are not masked at all: what they compute is not read,
      // and a full word costs the whole warp one comparison (mask_scores)
      int limit = 0x7fffffff;
      if (!SPARSE && rvalid) {
        const int Ls = p.seqlens[req];
        limit = Ls;
        if (p.causal) limit = Ls - p.s_q + row_query(p, pc.unit, grow) + 1;
      }
      float m_used = -INFINITY, l_sum = 0.f, scale_log2 = 0.f;  // scale_log2: of this row's raw scores
      int last_gt = -1;
      for (int k = pc.t0; k < pc.t1 && !stop; ++k, ++gt) {
        const int b = gt & 1;
        // validity of the 128 keys of this tile for this row (bit i of word w = key 32w + i)
        uint4 vmask;
        if (SPARSE) {
          const int d = gt % fp4::kRowDepth;
          if (!timed_wait_all(c, &rt->full[d], (gt / fp4::kRowDepth) & 1, p)) { stop = true; break; }
          vmask = *reinterpret_cast<const uint4*>(rt->valid[d]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&rt->empty[d]);
        } else {
          const int nv = dense_tile_valid(limit, k);
          auto word = [nv](int w) {
            const int nb = min(32, max(0, nv - 32 * w));
            return nb >= 32 ? 0xffffffffu : ((1u << nb) - 1u);
          };
          vmask = make_uint4(word(0), word(1), word(2), word(3));
        }
        if (!timed_wait_all(c, &c->s_full[b], (gt >> 1) & 1, p)) { stop = true; break; }
        tc_fence_after();
        if (k == pc.t0) scale_log2 = fp4::row_scale(p.scale_log2, c->q_back[pi & 1][r & 63]);
        const uint32_t s_addr = tmem + lane_base + kTmemS + 128 * b;
        // pass 1: tile max
        float tmax = -INFINITY;
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          uint32_t sv[32];
          tmem_ld32(s_addr + 32 * w, sv);
          tmem_ld_wait();
          fp4::mask_scores(sv, pick4u(vmask, w));
#pragma unroll
          for (int i = 0; i < 32; ++i) tmax = fmaxf(tmax, __uint_as_float(sv[i]));
        }
        float alpha = 1.f;
        int need = 0;
        if ((tmax - m_used) * scale_log2 > kRescaleLog2) {  // also for the first keys; never for -inf - -inf
          const float m_new = tmax;
          alpha = (m_used == -INFINITY) ? 0.f : ex2_approx((m_used - m_new) * scale_log2);
          need = rvalid && (k != pc.t0) && (m_used != -INFINITY);
          m_used = m_new;
          l_sum *= alpha;
        }
        // pass 2: probabilities (a masked score is -inf: e^-inf = 0) -> f16, staged
        // in TMEM over the S columns already read (tokens 32w.. -> columns 16w..)
        const float mc = m_used == -INFINITY ? 0.f : m_used;
        uint64_t sum = join2(0.f, 0.f);
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          uint32_t sv[32];
          tmem_ld32(s_addr + 32 * w, sv);
          tmem_ld_wait();
          fp4::mask_scores(sv, pick4u(vmask, w));
          uint32_t pk[16];
          fp4::probabilities(sv, mc, scale_log2, pk, sum);
          tmem_st16(s_addr + 16 * w, pk);
        }
        tmem_st_wait();
        float even, odd;
        split2(sum, even, odd);
        l_sum += even + odd;
        if (owner) c->alpha[r] = alpha;
        if (need) c->rescale_flag[gt & 1] = 1;
        if (!group_sync(c, &c->grp_sm, gph, p)) { stop = true; break; }
        const bool do_rescale = *(volatile int*)&c->rescale_flag[gt & 1] != 0;
        // the O MMAs of the previous tile must be complete before O^T is
        // rescaled and before P^T (which they read) is overwritten
        if (gt >= 1 && !timed_wait_all(c, &c->o_done, (gt - 1) & 1, p)) { stop = true; break; }
        tc_fence_after();
        if (do_rescale) {
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
#pragma unroll 1
            for (int c16 = 0; c16 < NR / 16; ++c16) {
              uint32_t ov[16];
              const uint32_t a = tmem + lane_base + 64 * m + 16 * c16;
              tmem_ld16(a, ov);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * c->alpha[16 * c16 + i]);
              tmem_st16(a, ov);
            }
          }
          tmem_st_wait();
          if (!group_sync(c, &c->grp_sm, gph, p)) { stop = true; break; }
          if (threadIdx.x == 128) c->rescale_flag[gt & 1] = 0;
        }
        // P^T, K-major [NR rows][128 tokens]: tokens 64h.. in slice h, 8 tokens per 16-B chunk
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          uint32_t pk[16];
          tmem_ld16(s_addr + 16 * w, pk);
          tmem_ld_wait();
          if (owner && r < NR) {
            uint8_t* rowp = sP + (w >> 1) * (NR * 128) + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int ch = 4 * (w & 1) + q;
              *reinterpret_cast<uint4*>(rowp + ((ch ^ (r & 7)) << 4)) =
                  make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&c->p_full);  // scores and staged probabilities of this buffer are consumed too
        last_gt = gt;
      }
      if (stop) break;
      // ---------------- epilogue of the piece
      if (last_gt >= 0 && !timed_wait_all(c, &c->o_done, last_gt & 1, p)) { stop = true; break; }
      tc_fence_after();
      if (owner) {
        float inv = 0.f, lse = -INFINITY;
        if (!(l_sum <= 0.f)) {  // NaN is no empty row: it goes into both results
          inv = 1.f / l_sum;
          lse = m_used * scale_log2 * 0.693147181f + logf(l_sum * fp4::kProbInv);
        }
        if (pc.single && rvalid && p.sink != nullptr) inv *= fold_sink(lse, p.sink[row_head(p, pc.unit, row0 + r)]);
        c->inv_l[r] = inv;
        if (rvalid) {
          const size_t grow_all = (size_t)pc.unit * p.rows + row0 + r;
          if (pc.single) p.lse[grow_all] = lse;
          else p.ws_lse[(size_t)pc.ws_idx * p.rows + row0 + r] = lse;
        }
      }
      if (!group_sync(c, &c->grp_sm, gph, p)) { stop = true; break; }
      // one pointer per piece and constant offsets from it: with the address and
      // the kind of output worked out per element this took 20 us a piece
      const size_t row_at = (size_t)(pc.single ? pc.unit : pc.ws_idx) * p.rows * kDv + 32 * q4 + lane;
      if (pc.single) store_rows<NR>(static_cast<__nv_bfloat16*>(p.out) + row_at, tmem + lane_base, c->inv_l, rows_here);
      else store_rows<NR>(p.ws_o + row_at, tmem + lane_base, c->inv_l, rows_here);
      tc_fence_before();
      if (!group_sync(c, &c->grp_sm, gph, p)) { stop = true; break; }
      mbar_arrive(&c->o_free);
      ++pi;
    }
  }

  // ---------------------------------------------------------------- teardown
  griddep_launch_dependents();  // the combine may be scheduled (it waits for this grid)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int NR, bool SPARSE>
cudaError_t launch_one(const CUtensorMap& tq, const DecodeParams& p, int parts, cudaStream_t stream) {
  constexpr int smem = Smem<NR>::total + 1024;
  auto kern = mla_decode_fp4_kernel<NR, SPARSE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(parts), dim3(fp4::kThreads), smem, stream, tq, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_fp4(const CUtensorMap& tq, const DecodeParams& p, int parts, bool sparse,
                              cudaStream_t stream) {
  // <= 16 rows run in the 32-row kernel: what the extra rows hold (P^T rows and
  // O^T columns of their own) is never stored. The rule is the row count: O's MMAs,
  // rescale and epilogue grow with NR. 48 rows in the 48-row kernel against the
  // 64-row one, us a step: 64 requests x 8192 tokens 182 / 184, x 40 rows x 4096
  // 108 / 109; 32 rows (ragged, 128 requests) in the 32-row kernel 410 / 412
  if (p.rows <= 32) return sparse ? launch_one<32, true>(tq, p, parts, stream) : launch_one<32, false>(tq, p, parts, stream);
  if (p.rows <= 48) return sparse ? launch_one<48, true>(tq, p, parts, stream) : launch_one<48, false>(tq, p, parts, stream);
  return sparse ? launch_one<64, true>(tq, p, parts, stream) : launch_one<64, false>(tq, p, parts, stream);
}

}  // namespace mla
