// Device code shared by the two decode kernels of the 4-bit cache
// (mla_decode_fp4.cu, mla_decode_fp4_pair.cu): the order of the operand ring,
// the warp that resolves cache rows, and the eight warps that turn 416-byte
// token records into tensor-core operands.
//
// A record is 256 bytes of E2M1 pairs, 32 UE4M3 scales (one per 16 latent
// values) and 64 bf16 RoPE dims. Latent values become bf16 without rounding:
// an E2M1 x UE4M3 product has at most 6 significant bits.
//
// Conversion: a nibble's three magnitude bits, put where a bf16 has the two
// low exponent bits and the top mantissa bit, read as its value times 2^-126
// (exponent field 0 is the subnormal 0.5); one multiplication by scale * 2^119
// gives value * 2^-7 and the sign bit is moved along, five instructions for
// two values. The 2^7 is put back in the query (K) and the output (V). Both
// halves of a 32-bit word are worked on at once, so the eight values of a word
// come out as elements 0 4 1 5 2 6 3 7: the query is put in the same order
// before its first use, and the output is written back in order.
// The five instructions bound the kernels: 142 clk of a 16 KB slot's ~256 clk
// of MMA time for eight warps alone on an SM, against 197 for byte-permute
// tables and 131 for the hardware conversion to f16, whose type Q lacks.
//
// Both operands use one kind of ring entry, 128 tokens x 128 latent dims as two
// 64-dim slices (32 KB): 64 contiguous code bytes of a token feed an entry, so
// four lanes share a line of the cache, and the L1 tag lookups (one a clock),
// which bounded 64-dim entries, halve. A converter thread stages the codes of
// its next entry in shared memory of its own (cp.async), scales one phase
// ahead in registers. Reading the codes again for V costs 256 bytes a token
// from L2, a quarter of the bf16 cache's V re-read.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_decode_util.cuh"

namespace mla {
namespace fp4 {

constexpr int kSlot = 32768;     // ring entry: two slices of 128 tokens x 64 dims
constexpr int kSlice = 16384;
constexpr int kN = 3;            // ring entries
constexpr int kGroups = 2;       // converter groups of four warps
constexpr int kCvWarps = 4 * kGroups;
constexpr int kRowDepth = 4;     // steps whose cache rows are resolved ahead
constexpr int kThreads = 256 + 32 * kCvWarps;
constexpr int kStageBytes = kGroups * 8192;  // the code bytes of one entry per group

// Order of a piece of n steps: phase h = 0 -> K of step 0; h = 2g+1 -> K of
// step g+1 (only if g+1 < n); h = 2g+2 -> V of step g. A K phase is five ring
// entries (four of latent dims, then the RoPE slice), a V phase four.
__device__ __forceinline__ bool phase_exists(int h, int nsteps) { return !((h & 1) && (h >> 1) + 1 >= nsteps); }
__device__ __forceinline__ bool phase_is_k(int h) { return h == 0 || (h & 1); }
__device__ __forceinline__ int phase_step(int h) { return h == 0 ? 0 : (h & 1) ? (h >> 1) + 1 : (h >> 1) - 1; }

// Steps of a piece: one 128-token tile (a single CTA) or two (a CTA pair).
template <bool PAIR>
__device__ __forceinline__ int steps_of(const Piece& pc) {
  return PAIR ? (pc.t1 - pc.t0 + 1) >> 1 : pc.t1 - pc.t0;
}

// Walks the phases of every piece of a part.
template <bool PAIR>
struct Phases {
  PieceIter it;
  Piece pc;
  int h = 0, nsteps = 0, step0 = 0;  // step0: index of the piece's first step among the part's steps
  bool in_piece = false;
  __device__ bool next() {
    if (in_piece) {
      do ++h;
      while (h <= 2 * nsteps && !phase_exists(h, nsteps));
      if (h <= 2 * nsteps) return true;
      step0 += nsteps;
    }
    in_piece = it.next(pc);
    if (!in_piece) return false;
    nsteps = steps_of<PAIR>(pc);
    h = 0;
    return true;
  }
  __device__ bool is_k() const { return phase_is_k(h); }
  __device__ int step() const { return step0 + phase_step(h); }
};

// Cache rows of the steps in flight (-1: past the request's end, outside the
// piece or an ignored index: converted to zeros), and with token-sparse
// indices the key validity bits (word w, bit i = key 32w + i of the step).
struct RowTable {
  uint64_t full[kRowDepth], empty[kRowDepth];
  int32_t row[kRowDepth][256];
  uint32_t valid[kRowDepth][8];
};

// Position in the ring: entry and the parity of its current use.
struct RingPos {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int n = 1) {
    slot += n;
    while (slot >= kN) {
      slot -= kN;
      parity ^= 1u;
    }
  }
  __device__ __forceinline__ RingPos at(int n) const {
    RingPos r = *this;
    r.advance(n);
    return r;
  }
};

// Eight bytes that are read once: no L1 line is kept for them.
__device__ __forceinline__ uint2 ldg8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// ---------------------------------------------------------------- conversions
// Eight E2M1 codes (one word, element i in nibble i) times a scale -> 8 bf16 in
// element order 0 4 1 5 2 6 3 7. s: the scale * 2^119, twice.
__device__ __forceinline__ uint4 e2m1x8(uint32_t w, __nv_bfloat162 s) {
  constexpr uint32_t kSign = 0x80008000u, kMag = 0x01C001C0u;
  uint32_t o[4] = {((w << 12) & kSign) | ((w << 6) & kMag), ((w << 8) & kSign) | ((w << 2) & kMag),
                   ((w << 4) & kSign) | ((w >> 2) & kMag), (w & kSign) | ((w >> 6) & kMag)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&o[i]), s);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Position within an 8-element group -> element.
__device__ __forceinline__ int element_of(int pos) { return (pos >> 1) | ((pos & 1) << 2); }
// A 16-byte chunk of the query: times 2^7, in the converted keys' order.
__device__ __forceinline__ uint4 order_query(uint4 v) {
  const __nv_bfloat162 f = __float2bfloat162_rn(128.f);
  uint32_t o[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                   __byte_perm(v.y, v.w, 0x7632)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&o[i]), f);
    o[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
constexpr float kOutScale = 128.f;  // what the converted V lacks

// Puts the latent slices of a query tile (64 rows) in order: thread t of `n`.
__device__ __forceinline__ void order_query_tile(uint8_t* q, int t, int n) {
#pragma unroll 4
  for (int i = t; i < 8 * 512; i += n) {  // chunk order within a slice does not matter
    uint4* c = reinterpret_cast<uint4*>(q) + i;
    *c = order_query(*c);
  }
}

// 32 codes and their two UE4M3 scale bytes (bit 7 ignored) -> chunks c0..c0+3
// of 128-byte row `row` of a swizzled tile.
__device__ __forceinline__ void store_item(uint4 codes, uint32_t scales, uint8_t* tile, int row, int c0) {
  const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(scales & 0x7F7Fu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
  const __nv_bfloat162 s0 = __float2bfloat162_rn(f.x * 0x1p119f), s1 = __float2bfloat162_rn(f.y * 0x1p119f);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(sw128(tile, row, c0 + i)) = e2m1x8(w[i], i < 2 ? s0 : s1);
}
// Copies a loaded word with an instruction that the compiler keeps where it is.
__device__ __forceinline__ uint32_t settle(uint32_t a) {
  uint32_t b;
  asm volatile("mov.b32 %0, %1;" : "=r"(b) : "r"(a));
  return b;
}

// Scores of 32 keys: those whose bit of `valid` is clear become -inf. Most
// words are full and cost one comparison.
__device__ __forceinline__ void mask_scores(uint32_t (&sv)[32], uint32_t valid) {
  if (valid == 0xffffffffu) return;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((valid >> i) & 1u)) sv[i] = 0xff800000u;
}

// ---------------------------------------------------------------- row warp
// One warp resolves the rows of every step of the part, up to kRowDepth steps
// ahead of the slowest reader. `wait(bar, parity)` is the kernel's bounded wait.
template <bool PAIR, bool SPARSE, class Wait>
__device__ __forceinline__ void row_warp(const DecodeParams& p, PieceIter it, RowTable* rt, int lane, Wait wait) {
  constexpr int kTok = PAIR ? 256 : 128;
  Piece pc;
  int gs = 0;
  bool stop = false;
  while (!stop && it.next(pc)) {
    const int req = unit_req(p, pc.unit);
    const int Ls = p.seqlens[req];
    const int npg = (Ls + kPage - 1) / kPage;
    const int n = steps_of<PAIR>(pc);
    for (int g = 0; g < n; ++g, ++gs) {
      const int d = gs % kRowDepth;
      bool ok = true;
      if (lane == 0) ok = wait(&rt->empty[d], ((gs / kRowDepth) & 1) ^ 1);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) { stop = true; break; }
      const int tok0 = (pc.t0 + (PAIR ? 2 : 1) * g) * kTile, end = min(pc.t1 * kTile, SPARSE ? p.topk : Ls);
#pragma unroll
      for (int w = 0; w < kTok / 32; ++w) {
        const int t = tok0 + 32 * w + lane;
        int row = -1;
        if (t < end) {
          if (SPARSE) row = sparse_row(p, pc.unit, t, true);
          else row = page_of(p, req, t / kPage, npg) * kPage + t % kPage;
        }
        rt->row[d][32 * w + lane] = row;
        if (SPARSE) {
          const uint32_t m = __ballot_sync(0xffffffffu, row >= 0);
          if (lane == 0) rt->valid[d][w] = m;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&rt->full[d]);
    }
  }
}

// ---------------------------------------------------------------- converters
// Fills the ring. Two groups of four warps take a phase's latent entries in
// turn (group g: entries g and g + 2) and its RoPE slice every other step. A
// thread converts four items of 32 codes per entry: tokens 32 w + 8 j +
// lane % 8, quarter lane / 8 of the entry's 128 dims; eight neighbouring lanes
// write the same chunk of eight rows, which the swizzle spreads over all banks.
// Entry e of a phase: K, and a single CTA's V: latent dims 128 e .. of the
// step's (own) tile; a pair's V: tile e / 2, value dims 256 (e % 2) + 128 rank ..
// `stage`: 16 bytes per item and thread.
// Scales: lane quarter q loads the eight scale bytes of entry q for its
// token, and an entry's are handed round by shuffle: one request a phase.
// The RoPE slice goes straight into its entry with cp.async, whose completion
// the entry's barrier counts.
// wait(bar, parity): the kernel's bounded wait; full(slot): the entry's barrier.
template <bool PAIR, class Wait, class Full>
__device__ __forceinline__ void convert_ring(const DecodeParams& p, const PieceIter& it, RowTable* rt, uint8_t* ring,
                                             uint4* stage, uint64_t* empty, int cw, int lane, int rank, Wait wait,
                                             Full full) {
  static_assert(kGroups == 2, "two entries per group and phase");
  const uint8_t* cache = static_cast<const uint8_t*>(p.kcache);
  const int grp = cw >> 2, w = cw & 3;
  const int tok = 32 * w + (lane & 7), q = lane >> 3;
  const int k0 = PAIR ? 128 * rank : 0;  // first token of this CTA's K tile
  stage += 32 * cw + lane;
  auto record = [&](bool k, int step, int e, int j) {
    return rt->row[step % kRowDepth][(k ? k0 : PAIR ? 128 * (e >> 1) : 0) + tok + 8 * j];
  };
  auto dim_of = [&](bool k, int e) { return PAIR && !k ? 256 * (e & 1) + 128 * rank : 128 * e; };
  auto fetch = [&](bool k, int step, int e) {
    const int off = dim_of(k, e) / 2 + 16 * q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = record(k, step, e, j);
      cp_async16(stage + j * (32 * kCvWarps), cache + (size_t)(row >= 0 ? row : 0) * kFp4RecordBytes + off,
                 row >= 0 ? 16u : 0u);
    }
    cp_async_commit();
  };
  auto scales = [&](bool k, int step, uint2 (&sc)[4]) {
    const int off = kFp4ScaleOff + dim_of(k, q) / 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = record(k, step, q, j);
      sc[j] = make_uint2(0, 0);
      if (row >= 0) sc[j] = ldg8(cache + (size_t)row * kFp4RecordBytes + off);
    }
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = true;
    if (lane == 0) ok = wait(bar, parity);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  };
  Phases<PAIR> nxt;     // the phase after the one being converted
  nxt.it = it;
  uint2 pre[4];         // its scales
  RingPos pos;          // first entry of the phase being converted
  bool have = nxt.next();
  if (have) {
    if (!wait_warp(&rt->full[0], 0)) return;
    scales(true, 0, pre);
    fetch(true, 0, grp);
  }
  bool stop = false;
  while (have && !stop) {
    const bool k = nxt.is_k();
    const int step = nxt.step();
    have = nxt.next();
    const bool nk = have && nxt.is_k();
    const int nstep = nxt.step();
    if (nk && !wait_warp(&rt->full[nstep % kRowDepth], (nstep / kRowDepth) & 1)) break;
    // one wait for all scales: loads share a few scoreboards, so one used
    // while younger loads are in flight would wait for those too
    uint2 sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sc[j] = make_uint2(settle(pre[j].x), settle(pre[j].y));
    if (have) scales(nk, nstep, pre);
    // not unrolled: the unrolled code left no room in the instruction cache
    // for the other roles
#pragma unroll 1
    for (int e = grp; e < 4; e += 2) {
      const RingPos at = pos.at(e);
      cp_async_wait<0>();
      uint4 codes[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) codes[j] = stage[j * (32 * kCvWarps)];
      if (e < 2) fetch(k, step, e + 2);
      else if (have) fetch(nk, nstep, grp);
      if (!wait_warp(&empty[at.slot], at.parity ^ 1u)) { stop = true; break; }
      uint8_t* s = ring + at.slot * kSlot + (q >> 1) * kSlice;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = __shfl_sync(0xffffffffu, sc[j].x, 8 * e + (lane & 7));
        const uint32_t hi = __shfl_sync(0xffffffffu, sc[j].y, 8 * e + (lane & 7));
        store_item(codes[j], (q & 2 ? hi : lo) >> (16 * (q & 1)), s, tok + 8 * j, 4 * (q & 1));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(at.slot));
    }
    if (stop) break;
    if (k) {
      if (grp == (step & 1)) {  // RoPE slice: 8 lanes per 128-byte row
        const RingPos at = pos.at(4);
        if (!wait_warp(&empty[at.slot], at.parity ^ 1u)) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = 32 * w + 4 * i + (lane >> 3), ch = lane & 7;
          const int row = rt->row[step % kRowDepth][k0 + t];
          cp_async16(sw128(ring + at.slot * kSlot, t, ch),
                     cache + (size_t)(row >= 0 ? row : 0) * kFp4RecordBytes + kFp4RopeOff + 16 * ch, row >= 0 ? 16u : 0u);
        }
        cp_async_mbar_arrive(full(at.slot));
        __syncwarp();
        if (lane == 0) mbar_arrive(full(at.slot));
      }
      pos.advance(5);
    } else {
      pos.advance(4);
    }
    // the rows of a step are last read by the fetches of its V phase: the one
    // of entry grp + 2 is issued in that phase itself
    if (!k) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&rt->empty[step % kRowDepth]);
    }
  }
  cp_async_wait<0>();  // no copy may land after the CTA has finished
}

}  // namespace fp4
}  // namespace mla
