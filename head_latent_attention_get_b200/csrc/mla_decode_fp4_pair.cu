// MLA decode over the 4-bit cache (MLA_KV_FP4_E2M1 records), units of 65-128
// query rows, paged or token-sparse: one CTA pair (cluster of 2 CTAs on two
// SMs) per scheduler part.
//
// Work split, TMEM layout and softmax are those of the bf16 pair kernel
// (mla_decode_pair.cu): a step is two 128-token tiles; CTA r supplies K of
// tile r and, for all 256 tokens, V of its value dims {256j + 128r + [0,128)}:
//   S = Q K^T   pair MMA M=128 (64 rows per CTA) x N=256 tokens x K=576
//   O = P V     pair MMA M=128 x N=256 value dims x K=256 tokens, twice
// Each CTA's ring is filled from the records
// (mla_fp4.cuh) in the order in which the even CTA's MMA issuer consumes it.
//
// Warp roles (640 threads per CTA):
//   0 Q via TMA (both CTAs)
//   1 TMEM allocation (both); MMA issue (even CTA); forwarding of the odd
//     CTA's slot completions (odd CTA)
//   2 cache rows   3 RoPE slices
//   4-7 softmax + epilogue (both): thread i = (row i % 64, token half i / 64)
//   8-11 raw copies   12-19 converters (and Q into form)
// All waits are bounded; a timeout sets MLA_DEVICE_STATUS_TIMEOUT, raises the
// abort flag of both CTAs, and every role winds down to the final cluster
// barrier, which both CTAs always reach.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mla_fp4.cuh"

namespace mla {
namespace fp4pair {

using fp4::kN;
constexpr int kQBytes = 9 * 8192;    // 64 rows x 576 dims
constexpr int kPBytes = 4 * 8192;    // 64 rows x 256 tokens (one buffer)
constexpr int kTmemCols = 512;
constexpr int kTmemS = 256;          // S buffers at columns 256 and 384; O at 0 and 128
constexpr float kRescaleLog2 = 8.0f;

struct Ctrl {
  // barriers counted on the even CTA (the MMA issuer) ...
  uint64_t q_full;                     // 16 arrivals: both CTAs' converter warps have Q in form
  uint64_t full[kN];                   // 4 arrivals here and the 4 bytes that the odd CTA's forwarder sends
  uint64_t p_full[2], o_free;          // 8 arrivals: 4 softmax warps x 2 CTAs
  uint64_t drain;
  // ... and in each CTA
  uint64_t q_raw;                      // Q as loaded
  uint64_t q_empty, empty[kN], rope_free;  // pair-MMA commits; rope_free: entry 1 of a K phase
  uint64_t s_full[2], o_done[2];       // pair-MMA commits; o_done[g & 1] completes O of step g
  uint64_t v_loc[kN];                  // odd CTA: the same 4 arrivals
  uint64_t grp_sm;                     // 128 softmax threads
  float q_back[2][64];                 // [piece parity][row]: what undoes the query's scaling
  uint32_t tmem_base;
  uint32_t forwarded;                  // where those 4 bytes land; never read
  int abort_flag;
  float mx[2][2][64];                  // [step parity][token half][row]: per-half tile max
  float lx[2][64];                     // [token half][row]: per-half row sum
};
static_assert(sizeof(Ctrl) <= 2560, "control block");

struct Smem {
  static constexpr int q = 0;
  static constexpr int ring = q + kQBytes;
  static constexpr int raw = ring + kN * fp4::kSlot;
  static constexpr int pt = (raw + fp4::kRaw * fp4::kRawBytes + 1023) / 1024 * 1024;  // swizzled
  static constexpr int ctrl = pt + kPBytes;
  static constexpr int rows = ctrl + 2560;
  static constexpr int total = rows + (int)sizeof(fp4::RowTable);
};
static_assert(Smem::total + 1024 <= 232448, "shared memory budget");

struct Pair {
  uint32_t rank;
  bool leader;
  Ctrl* c;
  uint32_t peer_abort;                 // cluster address of the other CTA's abort flag
};

__device__ __forceinline__ void raise_abort(const Pair& pr, const DecodeParams& p) {
  atomicOr(p.status, (uint32_t)MLA_DEVICE_STATUS_TIMEOUT);
  *(volatile int*)&pr.c->abort_flag = 1;
  st_cluster_u32(pr.peer_abort, 1u);
}

__device__ __forceinline__ bool aborted(const Pair& pr) { return *(volatile int*)&pr.c->abort_flag != 0; }

// Bounded wait with cluster-scope acquire (several barriers receive arrivals
// from the other CTA or pair-MMA commits).
__device__ __forceinline__ bool pwait(const Pair& pr, uint64_t* bar, uint32_t parity, const DecodeParams& p) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  if (aborted(pr)) return false;
  if (mbar_wait_cluster(bar, parity, p.timeout_ns)) return true;
  raise_abort(pr, p);
  return false;
}

// For all lanes of a warp that goes on to collective instructions: either all of
// them go on or, if the limit ran out for one, none.
__device__ __forceinline__ bool pwait_all(const Pair& pr, uint64_t* bar, uint32_t parity, const DecodeParams& p) {
  return __all_sync(0xffffffffu, pwait(pr, bar, parity, p)) != 0;
}

__device__ __forceinline__ bool group_sync(const Pair& pr, uint32_t& phase, const DecodeParams& p) {
  mbar_arrive(&pr.c->grp_sm);
  const bool ok = pwait_all(pr, &pr.c->grp_sm, phase & 1, p);
  ++phase;
  return ok;
}

// Arrive on barrier `bar` of the even CTA (a local arrive there, a remote one from the odd CTA).
__device__ __forceinline__ void arrive_leader(const Pair& pr, uint64_t* bar) {
  if (pr.leader) mbar_arrive(bar);
  else mbar_arrive_cluster(map_to_rank(smem_u32(bar), 0));
}

template <bool SPARSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(fp4::kThreads, 1)
    mla_decode_fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + Smem::q;
  uint8_t* sRing = smem + Smem::ring;
  uint8_t* sRaw = smem + Smem::raw;
  uint8_t* sP = smem + Smem::pt;
  Ctrl* c = reinterpret_cast<Ctrl*>(smem + Smem::ctrl);
  fp4::RowTable* rt = reinterpret_cast<fp4::RowTable*>(smem + Smem::rows);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: known to be uniform
  Pair pr;
  pr.rank = cluster_rank();
  pr.leader = pr.rank == 0;
  pr.c = c;
  pr.peer_abort = map_to_rank(smem_u32(&c->abort_flag), pr.rank ^ 1u);
  const int part = blockIdx.x >> 1;
  const int row0 = 64 * (int)pr.rank;   // first row of this CTA within a unit

  if (threadIdx.x == 0) {
    mbar_init(&c->q_full, 2 * fp4::kCvWarps);
    mbar_init(&c->q_raw, 1);
    for (int i = 0; i < kN; ++i) mbar_init(&c->full[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&c->p_full[i], 8);
    mbar_init(&c->o_free, 8);
    mbar_init(&c->drain, 1);
    mbar_init(&c->q_empty, 1);
    mbar_init(&c->rope_free, 1);
    for (int i = 0; i < kN; ++i) mbar_init(&c->empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&c->s_full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&c->o_done[i], 1);
    for (int i = 0; i < kN; ++i) mbar_init(&c->v_loc[i], 4);
    for (int i = 0; i < fp4::kRowDepth; ++i) {
      mbar_init(&rt->full[i], 1);
      mbar_init(&rt->empty[i], fp4::kLdWarps + 1 + (SPARSE ? 4 : 0));
    }
    for (int i = 0; i < fp4::kRaw; ++i) {
      mbar_init(&rt->raw_full[i], 32 * fp4::kLdWarps);
      mbar_init(&rt->raw_empty[i], 4);
    }
    mbar_init(&c->grp_sm, 128);
    c->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_q);
  if (warp == 1) {
    tmem_alloc_pair(&c->tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // barriers initialised and TMEM allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;
  griddep_wait();  // the scheduler's output (and every input) is ready

  PieceIter it;
  it.init(p, part);
  Piece pc;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return pwait(pr, bar, parity, p); };
  auto full = [&](int slot) { return pr.leader ? &c->full[slot] : &c->v_loc[slot]; };
  auto arrive = [&](int slot, int w) {  // one of an entry's four arrivals
    if (pr.leader && w == 0) mbar_arrive_expect_tx(&c->full[slot], 4);
    else mbar_arrive(full(slot));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ Q
    if (lane == 0) {
      int pi = 0, q_issued = 0;
      while (it.next(pc)) {
        if (!pwait(pr, &c->q_empty, (pi & 1) ^ 1, p)) break;
        mbar_arrive_expect_tx(&c->q_raw, kQBytes);
        for (int j = 0; j < 9; ++j) tma_load_2d(sQ + j * 8192, &tm_q, &c->q_raw, 64 * j, pc.unit * p.rows + row0);
        ++q_issued;
        ++pi;
      }
      if (q_issued > 0) mbar_wait(&c->q_raw, (uint32_t)((q_issued - 1) & 1), p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 2) {
    fp4::row_warp<true, SPARSE>(p, it, rt, lane, (int)pr.rank, wait);
  } else if (warp == 3) {
    fp4::load_rope<true>(p, it, rt, sRing, &c->rope_free, lane, (int)pr.rank, wait, full, arrive);
  } else if (warp >= 8 && warp < 12) {
    fp4::load_raw<true>(p, it, rt, sRaw, warp - 8, lane, (int)pr.rank, wait);
  } else if (warp >= 12) {
    fp4::convert_ring<true>(it, rt, sRing, sRaw, c->empty, warp - 12, lane, wait, arrive, [&](int piece) {
      if (!fp4::wait_warp(&c->q_raw, piece & 1, wait)) return false;
      fp4::scale_query_rows(sQ, c->q_back[piece & 1], min(64, p.rows - row0), warp - 12, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_leader(pr, &c->q_full);
      return true;
    });
  } else if (warp == 1 && !pr.leader) {
    // ------------------------------------------------------------ odd CTA: forward slot completions
    if (lane == 0) {
      int sc = 0;
      bool stop = false;
      while (!stop && it.next(pc)) {
        const int nslots = 9 * fp4::steps_of<true>(pc);  // 5 K and 4 V entries per step
        for (int i = 0; i < nslots; ++i, ++sc) {
          if (!pwait(pr, &c->v_loc[sc % kN], (sc / kN) & 1, p)) { stop = true; break; }
          // RoPE comes by cp.async: entry 4 of the piece's first K phase, 9, 18, .. of the others
          if (i == 4 || (i > 0 && i % 9 == 0)) fence_proxy_async_smem();
          // The rows (acquired from v_loc, fenced by their writers or above) must
          // come before the even CTA's use of them: the count of an asynchronous
          // store is a release at cluster scope. 64 x 128 x 4096 tokens, us a call when
          // it was added: 137 (134 with a relaxed arrive, which orders nothing; 144
          // with arrive.release.cluster, 147 with that in the converters themselves)
          st_async_u32(map_to_rank(smem_u32(&c->forwarded), 0), 0, map_to_rank(smem_u32(&c->full[sc % kN]), 0));
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: S(0), S(1), O(0), S(2), O(1), ...
    const uint32_t idesc_s = idesc_f16(128, 256, false, false), idesc_r = idesc_bf16(128, 256, false, false);
    const uint32_t idesc_o = idesc_f16(128, 256, false, true);
    // descriptors: Q, K and P are K-major, V is MN-major (slices 16 KB apart)
    const uint32_t q_lo = sdesc_lo(smem_u32(sQ), 16), k_lo = sdesc_lo(smem_u32(sRing), 16);
    const uint32_t v_lo = sdesc_lo(smem_u32(sRing), fp4::kSlice), p_lo = sdesc_lo(smem_u32(sP), 16);
    constexpr uint32_t d_hi = sdesc_hi(1024);
    int gs = 0, go = 0, pi = 0;
    fp4::RingPos pos;
    bool stop = false;
    if (elect_one()) {
      while (!stop && it.next(pc)) {
        if (!pwait(pr, &c->q_full, pi & 1, p)) { stop = true; break; }
        const int nsteps = fp4::steps_of<true>(pc);
        for (int h = 0; h <= 2 * nsteps && !stop; ++h) {
          if (!fp4::phase_exists(h, nsteps)) continue;
          const int g = fp4::phase_step(h);
          if (fp4::phase_is_k(h)) {
            // S buffer b was last read by the softmax of step gs - 2, whose
            // P the O product of step gs - 2 (issued just before) waited for
            const int b = gs & 1;
            tc_fence_after();
            const uint32_t d = tmem + kTmemS + 128 * b;
            for (int e = 0; e < 5; ++e, pos.advance()) {  // four latent entries of two slices, then RoPE
              const int slot = pos.slot;
              if (!pwait(pr, &c->full[slot], pos.parity, p)) { stop = true; break; }
              if (e == 4) fence_proxy_async_smem();  // RoPE comes by cp.async
              tc_fence_after();
              const uint32_t qa = q_lo + 2 * e * (8192 >> 4), kb = k_lo + slot * (fp4::kSlot >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                if (kk < 4 || e < 4)
                  mma_bf16_ss_pair(d, sdesc_join(qa + (kk >> 2) * (8192 >> 4) + (kk & 3) * 2, d_hi),
                                   sdesc_join(kb + (kk >> 2) * (fp4::kSlice >> 4) + (kk & 3) * 2, d_hi), e < 4 ? idesc_s : idesc_r,
                                   (e | kk) != 0 ? 1u : 0u);
              mma_commit_pair(&c->empty[slot]);
              if (e == 1) mma_commit_pair(&c->rope_free);
            }
            if (stop) break;
            if (!(gs == 0 && (p.debug_flags & MLA_DEBUG_WITHHOLD_SCORES))) mma_commit_pair(&c->s_full[b]);
            ++gs;
            if (g == nsteps - 1) mma_commit_pair(&c->q_empty);  // Q is free once the last S completes
          } else {
            const bool first = g == 0;
            if (first && pi > 0 && !pwait(pr, &c->o_free, (pi - 1) & 1, p)) { stop = true; break; }
            if (!pwait(pr, &c->p_full[go & 1], (go >> 1) & 1, p)) { stop = true; break; }
            for (int e = 0; e < 4; ++e, pos.advance()) {  // tile e / 2, value dims 256 (e % 2) ..
              const int slot = pos.slot;
              if (!pwait(pr, &c->full[slot], pos.parity, p)) { stop = true; break; }
              tc_fence_after();
              const uint32_t va = v_lo + slot * (fp4::kSlot >> 4), pa = p_lo + (e >> 1) * (16384 >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ss_pair(tmem + 128 * (e & 1), sdesc_join(pa + (kk >> 2) * (8192 >> 4) + (kk & 3) * 2, d_hi),
                                 sdesc_join(va + kk * (2048 >> 4), d_hi), idesc_o, (first && e < 2 && kk == 0) ? 0u : 1u);
              mma_commit_pair(&c->empty[slot]);
            }
            if (stop) break;
            mma_commit_pair(&c->o_done[go & 1]);
            ++go;
          }
        }
        ++pi;
      }
      mma_commit_pair(&c->drain);  // every MMA this thread issued has completed before teardown
      mbar_wait(&c->drain, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ softmax + epilogue
    const int ti = threadIdx.x - 128;                     // TMEM lane of this thread
    const int row = ti & 63, half = ti >> 6;
    const int grow = row0 + row;                          // row within the unit
    const bool rvalid = grow < p.rows;
    const uint32_t lane_base = (uint32_t)(32 * (warp - 4)) << 16;
    uint32_t gph = 0;
    int gt = 0, pi = 0;
    bool stop = false;
    while (!stop && it.next(pc)) {
      const int req = unit_req(p, pc.unit);
      const int Ls = p.seqlens[req];
      const int limit = p.causal ? Ls - p.s_q + row_query(p, pc.unit, grow) + 1 : Ls;
      float m_used = -INFINITY, l_sum = 0.f, scale_log2 = 0.f;  // scale_log2: of this row's raw scores
      int last_gt = -1;
      for (int k = pc.t0; k < pc.t1 && !stop; k += 2, ++gt) {
        const int b = gt & 1;
        // validity of this thread's 128 keys: bit i of word w = key 32w + i
        uint4 vm;
        if (SPARSE) {
          const int d = gt % fp4::kRowDepth;
          if (!pwait_all(pr, &rt->full[d], (gt / fp4::kRowDepth) & 1, p)) { stop = true; break; }
          vm = rvalid ? *reinterpret_cast<const uint4*>(&rt->valid[d][4 * half]) : make_uint4(0, 0, 0, 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(&rt->empty[d]);
        } else {
          const int tile = k + half;
          const int nv = (rvalid && tile < pc.t1) ? dense_tile_valid(limit, tile) : 0;
          auto word = [nv](int w) {
            const int nb = min(32, max(0, nv - 32 * w));
            return nb >= 32 ? 0xffffffffu : ((1u << nb) - 1u);
          };
          vm = make_uint4(word(0), word(1), word(2), word(3));
        }
        if (!pwait_all(pr, &c->s_full[b], (gt >> 1) & 1, p)) { stop = true; break; }
        tc_fence_after();
        if (k == pc.t0) scale_log2 = fp4::row_scale(p.scale_log2, c->q_back[pi & 1][row]);
        const uint32_t s_addr = tmem + lane_base + kTmemS + 128 * b;
        // pass 1: max over this thread's 128 keys
        float tmax = -INFINITY;
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          uint32_t sv[32];
          tmem_ld32(s_addr + 32 * w, sv);
          tmem_ld_wait();
          fp4::mask_scores(sv, pick4u(vm, w));
#pragma unroll
          for (int i = 0; i < 32; ++i) tmax = fmaxf(tmax, __uint_as_float(sv[i]));
        }
        c->mx[gt & 1][half][row] = tmax;
        if (!group_sync(pr, gph, p)) { stop = true; break; }
        tmax = fmaxf(tmax, c->mx[gt & 1][half ^ 1][row]);
        // both threads of a row take the same decision from the same values
        float alpha = 1.f;
        bool need = false;
        if ((tmax - m_used) * scale_log2 > kRescaleLog2) {  // also for the first keys; never for -inf - -inf
          alpha = (m_used == -INFINITY) ? 0.f : ex2_approx((m_used - tmax) * scale_log2);
          need = (k != pc.t0) && (m_used != -INFINITY);
          m_used = tmax;
          l_sum *= alpha;
        }
        // pass 2: probabilities (a masked score is -inf: e^-inf = 0) -> f16 -> the P buffer,
        // K-major [64 rows][64 keys] per slice: keys 64s.. in slice s; this
        // thread's keys are 128*half + [0,128), slices 2*half and 2*half + 1.
        // The single P buffer was last read by the O product of step gt - 1,
        // which must also be complete before O is rescaled. (O of step gt + 1,
        // the next completion of the same barrier, needs this thread's P, so
        // the parity wait never falls two phases behind.) The first
        // quarter is computed into registers while that product runs.
        const float mc = m_used == -INFINITY ? 0.f : m_used;
        uint64_t sum = join2(0.f, 0.f);
        auto probs = [&](int w, uint32_t (&pk)[16]) {
          uint32_t sv[32];
          tmem_ld32(s_addr + 32 * w, sv);
          tmem_ld_wait();
          fp4::mask_scores(sv, pick4u(vm, w));
          fp4::probabilities(sv, mc, scale_log2, pk, sum);
        };
        auto store = [&](int w, const uint32_t (&pk)[16]) {
          uint8_t* rowp = sP + (2 * half + (w >> 1)) * 8192 + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int ch = 4 * (w & 1) + q;
            *reinterpret_cast<uint4*>(rowp + ((ch ^ (row & 7)) << 4)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          }
        };
        uint32_t pk[16];
        probs(0, pk);
        if (gt >= 1 && !pwait_all(pr, &c->o_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, p)) { stop = true; break; }
        store(0, pk);
#pragma unroll 1
        for (int w = 1; w < 4; ++w) {
          probs(w, pk);
          store(w, pk);
        }
        tc_fence_after();
        float even, odd;
        split2(sum, even, odd);
        l_sum += even + odd;
        // A warp's rows grow apart, but its tensor-memory accesses are collective:
        // all of its rows are multiplied as soon as one needs it (alpha is 1 for the others).
        if (__any_sync(0xffffffffu, need)) {
          // O holds every product up to step gt - 1 (waited for above)
#pragma unroll 1
          for (int c16 = 0; c16 < 16; ++c16) {  // 2 x 128 columns of this row
            uint32_t ov[16];
            const uint32_t a = tmem + lane_base + 16 * c16;
            tmem_ld16(a, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st16(a, ov);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(pr, &c->p_full[b]);  // P written, O rescaled, scores consumed
        last_gt = gt;
      }
      if (stop) break;
      // ---------------- epilogue of the piece
      c->lx[half][row] = l_sum;
      if (!group_sync(pr, gph, p)) { stop = true; break; }
      const float l_tot = l_sum + c->lx[half ^ 1][row];
      if (last_gt >= 0 && !pwait_all(pr, &c->o_done[last_gt & 1], (last_gt >> 1) & 1, p)) { stop = true; break; }
      tc_fence_after();
      float inv = 0.f, lse = -INFINITY;
      if (!(l_tot <= 0.f)) {  // NaN is no empty row: it goes into both results
        inv = 1.f / l_tot;
        lse = m_used * scale_log2 * 0.693147181f + logf(l_tot * fp4::kProbInv);
      }
      if (pc.single && rvalid && p.sink != nullptr) inv *= fold_sink(lse, p.sink[row_head(p, pc.unit, grow)]);
      const size_t orow = (size_t)pc.unit * p.rows + grow;
      if (rvalid && half == 0) {
        if (pc.single) p.lse[orow] = lse;
        else p.ws_lse[(size_t)pc.ws_idx * p.rows + grow] = lse;
      }
#pragma unroll 1
      for (int jd = 0; jd < 2; ++jd) {
        const int d0 = 256 * jd + 128 * half;
#pragma unroll 1
        for (int c16 = 0; c16 < 8; ++c16) {
          uint32_t ov[16];
          tmem_ld16(tmem + lane_base + 128 * jd + 16 * c16, ov);
          tmem_ld_wait();
          if (rvalid) {
            if (pc.single) {
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                pk[i] = pack_bf16x2(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * kDv + d0 + 16 * c16);
              dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            } else {
              float4* dst = reinterpret_cast<float4*>(p.ws_o + ((size_t)pc.ws_idx * p.rows + grow) * kDv + d0 + 16 * c16);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_float4(__uint_as_float(ov[4 * i]) * inv, __uint_as_float(ov[4 * i + 1]) * inv,
                                     __uint_as_float(ov[4 * i + 2]) * inv,
                                     __uint_as_float(ov[4 * i + 3]) * inv);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(pr, &c->o_free);
      ++pi;
    }
  }

  // ---------------------------------------------------------------- teardown
  // Every copy of this CTA has landed: the loader, RoPE and Q warps waited
  // for their own. After an abort a remote arrive or a pair MMA of the other
  // CTA may be pending for microseconds, so the CTA holds its shared memory
  // for a fixed 200 us of wall time (%globaltimer, not a sleep hint that may
  // return early) before the final cluster barrier.
  if (aborted(pr)) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000) {
    }
  }
  griddep_launch_dependents();  // the combine may be scheduled (it waits for this grid)
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no pair MMA, copy or remote arrive of either CTA is still pending
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace fp4pair

cudaError_t launch_decode_fp4_pair(const CUtensorMap& tq, const DecodeParams& p, int parts, bool sparse,
                                   cudaStream_t stream) {
  constexpr int smem = fp4pair::Smem::total + 1024;
  auto kern = sparse ? fp4pair::mla_decode_fp4_pair_kernel<true> : fp4pair::mla_decode_fp4_pair_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(2 * parts), dim3(fp4::kThreads), smem, stream, tq, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
