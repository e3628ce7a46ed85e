// Device code shared by the two decode kernels of the 4-bit cache
// (mla_decode_fp4.cu, mla_decode_fp4_pair.cu): the order of the operand ring,
// the warp that resolves cache rows, and the eight warps that turn 416-byte
// token records into tensor-core operands.
//
// A record is 256 bytes of E2M1 pairs, 32 UE4M3 scales (one per 16 latent
// values) and 64 bf16 RoPE dims. Latent values become f16, without rounding: an
// E2M1 x UE4M3 product has at most 6 significant bits and lies in [2^-10, 2688].
// The hardware turns a byte of codes into two f16, which one multiplication
// scales: 11 instructions for eight values, against 17 (integer shifts and
// masks) or 19 (byte-permute tables) for bf16. One MMA wants one type for both
// operands, so the query's latent part is f16 too, each row times a power of
// two that puts its largest value at 2^11..2^12: what an f16 then cannot hold
// is below 2^-36 of it, far under the fp32 accumulation. The RoPE part stays
// bf16 on both sides (times the same power), in MMAs of its own into the same
// accumulator, which RoPE keys up to 2^100 cannot overflow (64 x 2^12 x 2^100).
// Probabilities are f16.
//
// Both operands use one kind of ring entry, 128 tokens x 128 latent dims as two
// 64-dim slices (32 KB): 64 contiguous code bytes of a token feed an entry, so
// four lanes share a line of the cache, and the L1 tag lookups (one a clock)
// are half of those of 64-dim entries. Reading the codes again for V costs 256
// bytes a token from L2, a quarter of the bf16 cache's V re-read.
//
// The work is cut by latency: one warp resolves rows, four copy raw bytes, one
// the RoPE slices, eight only convert (two groups on alternate entries), so no
// role waits for another's round trips (with the raw copies in the converter
// warps 64 x 64 heads x 8192 tokens took 219 us in place of 205).
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
constexpr int kLdWarps = 4;
constexpr int kThreads = 256 + 32 * (kLdWarps + kCvWarps);
constexpr int kRaw = 2;                    // raw buffers: 8 KB of codes, 1 KB of scales
constexpr int kRawBytes = 8192 + 1024;

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
  uint64_t full[kRowDepth], empty[kRowDepth];  // empty: loader warps, the RoPE warp (and, sparse, the softmax warps)
  uint64_t raw_full[kRaw], raw_empty[kRaw];    // 128 loader threads; 4 converter warps
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

// ---------------------------------------------------------------- conversions
// Eight E2M1 codes (one word, element i in nibble i) times a scale -> 8 f16.
__device__ __forceinline__ uint4 e2m1x8(uint32_t w, __half2 s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((w >> (8 * i)) & 0xFFu), __NV_E2M1);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&hr), s);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// 32 codes and their two UE4M3 scale bytes (bit 7 ignored) -> chunks c0..c0+3
// of 128-byte row `row` of a swizzled tile.
__device__ __forceinline__ void store_item(uint4 codes, uint32_t scales, uint8_t* tile, int row, int c0) {
  const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(scales & 0x7F7Fu), __NV_E4M3);
  const __half2 sc = *reinterpret_cast<const __half2*>(&hr);
  const __half2 s0 = __low2half2(sc), s1 = __high2half2(sc);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(sw128(tile, row, c0 + i)) = e2m1x8(w[i], i < 2 ? s0 : s1);
}

// ---------------------------------------------------------------- query
// Puts a query tile (nine 64-row slices of bf16 as TMA wrote them) into the
// form above: this warp rows 8 cw .. below `rows`, half a warp per row. back[row]: the row's power of two
// undone, which the softmax multiplies into its scale.
__device__ __forceinline__ void scale_query_rows(uint8_t* q, float* back, int rows, int cw, int lane) {
  const int half = lane >> 4, l = lane & 15;
#pragma unroll 1
  for (int r0 = 8 * cw; r0 < min(8 * cw + 8, rows); r0 += 2) {
    const int row = r0 + half;
    // chunks l + 16 i of the row's 72 (slice, chunk): i < 4 latent, i = 4 (l < 8) RoPE
    uint4 v[5];
    uint32_t top = 0;  // largest magnitude: bf16 bits order like the values
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (i < 4 || l < 8) v[i] = *reinterpret_cast<const uint4*>(q + (2 * i + (l >> 3)) * 8192 + row * 128 + 16 * (l & 7));
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 2^e with e = 11 - exponent(top), kept where 2^e and 2^-e are normal floats
    const int e = top == 0 ? 0 : max(-126, min(126, 138 - (int)(top >> 7)));
    const float f = __uint_as_float((uint32_t)(127 + e) << 23);
    if (l == 0) back[row] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      if (i == 4 && l >= 8) break;
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]));
        w[j] = i < 4 ? pack_f16x2(x.x * f, x.y * f) : pack_bf16x2(x.x * f, x.y * f);
      }
      *reinterpret_cast<uint4*>(q + (2 * i + (l >> 3)) * 8192 + row * 128 + 16 * (l & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Factor of a row's raw scores in the exponent. Kept above 0, which would make
// a masked -inf a NaN; a row that the bound changes has scores below 2^-90.
__device__ __forceinline__ float row_scale(float scale_log2, float back) { return fmaxf(scale_log2 * back, 0x1p-126f); }

// Scores of 32 keys: those whose bit of `valid` is clear become -inf. Most
// words are full and cost one comparison.
__device__ __forceinline__ void mask_scores(uint32_t (&sv)[32], uint32_t valid) {
  if (valid == 0xffffffffu) return;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((valid >> i) & 1u)) sv[i] = 0xff800000u;
}

// Probabilities of 32 keys from their scores: 2^((s - m) * scale_log2 + 7), as
// f16 pairs, and their sums added to `sum` (even and odd keys). The difference is
// taken first: a product rounded before it would be off by more than 1 for
// scores past 2^24. A masked score is -inf: e^-inf = 0.
// The 7: the largest is then 2^7 and, before O is rescaled, 2^15 of f16's 65504 at
// most, and those down to 2^-21 of the largest keep f16's 11 bits, down to 2^-31
// some. Without it 2^-25 was 0 in the product with V but not in the sum, up to
// 2^-8 of the output at 128K keys. The sum has the same factor, so that it cancels
// in the output; the log-sum-exp takes it out. Times are the same.
constexpr float kProbLog2 = 7.0f, kProbInv = 0.0078125f;
__device__ __forceinline__ void probabilities(const uint32_t (&sv)[32], float m, float scale_log2, uint32_t (&pk)[16],
                                              uint64_t& sum) {
  const uint64_t nm = join2(-m, -m), sl = join2(scale_log2, scale_log2), up = join2(kProbLog2, kProbLog2);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    split2(fma2(add2(join2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), nm), sl, up), x0, x1);
    x0 = ex2_approx(x0);
    x1 = ex2_approx(x1);
    pk[i] = pack_f16x2(x0, x1);
    sum = add2(sum, join2(x0, x1));
  }
}

// ---------------------------------------------------------------- row warp
// One warp resolves the rows of every step of the part, up to kRowDepth steps
// ahead of the slowest reader. `wait(bar, parity)` is the kernel's bounded wait.
template <bool PAIR, bool SPARSE, class Wait>
__device__ __forceinline__ void row_warp(const DecodeParams& p, PieceIter it, RowTable* rt, int lane, int rank, Wait wait) {
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
      __syncwarp();
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) { stop = true; break; }
      const int tok0 = (pc.t0 + (PAIR ? 2 : 1) * g) * kTile, end = min(pc.t1 * kTile, SPARSE ? p.topk : Ls);
      // Sparse: all loads of a kind before the first use of one, so that a step
      // costs two round trips, not two per 32 tokens (32 requests x 128 heads x
      // 2048 selected tokens: 63 -> 51 us). Dense pairs lost by it (64 x 128 x
      // 4096: 122 -> 128 us): their prefetches then left in one burst.
      int pos[kTok / 32], page[kTok / 32];
      if (SPARSE) {
#pragma unroll
        for (int w = 0; w < kTok / 32; ++w) {
          const int t = tok0 + 32 * w + lane;
          pos[w] = t < end ? p.indices[(size_t)pc.unit * p.topk + t] : -1;
        }
#pragma unroll
        for (int w = 0; w < kTok / 32; ++w) {
          page[w] = -1;
          if (pos[w] >= 0 && pos[w] < Ls && pos[w] / kPage < p.bt_stride) page[w] = p.block_table[(size_t)req * p.bt_stride + pos[w] / kPage];
        }
      }
#pragma unroll
      for (int w = 0; w < kTok / 32; ++w) {
        const int t = tok0 + 32 * w + lane;
        int row = -1;
        if (SPARSE) {
          if (page[w] >= 0 && page[w] < p.num_pages) row = page[w] * kPage + pos[w] % kPage;
          else if (pos[w] != -1) atomicOr(p.status, (uint32_t)MLA_DEVICE_STATUS_BOUNDS);
        } else if (t < end) {
          row = page_of(p, req, t / kPage, npg) * kPage + t % kPage;
        }
        rt->row[d][32 * w + lane] = row;
        // the copies find the records in L2: whole pages, or a token's four lines
        const uint8_t* rec = static_cast<const uint8_t*>(p.kcache) + (size_t)(row >= 0 ? row : 0) * kFp4RecordBytes;
        if (!PAIR || (w >> 2) == rank) {
          if (SPARSE) {
            if (row >= 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(rec + min(128 * i, kFp4RecordBytes - 1)));
            }
          } else if (lane == 0 && !(w & 1) && row >= 0) {
            prefetch_l2(rec, min(kPage, Ls - t) * kFp4RecordBytes);
          }
        }
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

// All lanes wait, so that what they read next is ordered for each of them; a shuffle
// of one lane's outcome orders no memory. Decode and combine, us, 64 x 128 x 4096 /
// 64 x 64 x 8192 / ragged 16 heads / 32 x 128 topk 2048: 121 / 172 / 376 / 49; one
// lane waiting, with a warp barrier 131 / 177 / 372 / 50, without it 131 / 173 / 367 / 50.
template <class Wait>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Wait wait) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || __all_sync(0xffffffffu, wait(bar, parity));
}

// Entry e of a phase. K, and a single CTA's V: latent dims 128 e .. of the
// step's (own) tile; a pair's V: tile e / 2, value dims 256 (e % 2) + 128 rank ..
template <bool PAIR>
__device__ __forceinline__ int entry_token(bool k, int e, int rank) {
  return PAIR ? 128 * (k ? rank : e >> 1) : 0;
}
template <bool PAIR>
__device__ __forceinline__ int entry_dim(bool k, int e, int rank) {
  return PAIR && !k ? 256 * (e & 1) + 128 * rank : 128 * e;
}

// ---------------------------------------------------------------- loaders
// Four warps copy the raw bytes of the entries in order: warp w the 32 tokens
// 32 w .., four lanes on the 64 code bytes of a token, one on its 8 scale bytes.
template <bool PAIR, class Wait>
__device__ __forceinline__ void load_raw(const DecodeParams& p, const PieceIter& it, RowTable* rt, uint8_t* raw, int w,
                                         int lane, int rank, Wait wait) {
  const uint8_t* cache = static_cast<const uint8_t*>(p.kcache);
  Phases<PAIR> ph;
  ph.it = it;
  uint32_t n = 0;
  bool stop = false;
  while (!stop && ph.next()) {
    const bool k = ph.is_k();
    const int step = ph.step(), d = step % kRowDepth;
    if (k && !wait_warp(&rt->full[d], (step / kRowDepth) & 1, wait)) break;
#pragma unroll 1
    for (int e = 0; e < 4; ++e, ++n) {
      const int r = n % kRaw;
      if (!wait_warp(&rt->raw_empty[r], ((n / kRaw) & 1) ^ 1, wait)) { stop = true; break; }
      const int32_t* rows = rt->row[d] + entry_token<PAIR>(k, e, rank) + 32 * w;
      const int d0 = entry_dim<PAIR>(k, e, rank);
      uint8_t* buf = raw + r * kRawBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = rows[8 * j + (lane & 7)];
        cp_async16(buf + ((4 * w + j) * 32 + lane) * 16,
                   cache + (size_t)(row >= 0 ? row : 0) * kFp4RecordBytes + d0 / 2 + 16 * (lane >> 3), row >= 0 ? 16u : 0u);
      }
      const int row = rows[lane];
      cp_async8(buf + 8192 + (32 * w + lane) * 8,
                cache + (size_t)(row >= 0 ? row : 0) * kFp4RecordBytes + kFp4ScaleOff + d0 / 16, row >= 0 ? 8u : 0u);
      cp_async_mbar_arrive_noinc(&rt->raw_full[r]);
    }
    if (!stop && !k) {  // a step's rows are last read by its V phase
      __syncwarp();
      if (lane == 0) mbar_arrive(&rt->empty[d]);
    }
  }
  cp_async_wait_all();  // no copy may land after the CTA has finished, also where a wait above gave up
}

// ---------------------------------------------------------------- RoPE
// One warp copies the RoPE slice of every K phase straight into its ring entry,
// 8 lanes per 128-byte row. The entry's barrier counts the copies and, in the
// place of a converter group's four warps, four arrivals. cp.async writes like
// an ordinary store, and who waits for the entry fences it for the tensor core
// (64 x 128 x 4096 tokens: 124 -> 126 us by that fence in the odd CTA and 122 ->
// 124 by the issuer's; waiting and fencing here 129; two warps that hold the
// bytes in registers until the place is free 128, and 64 x 64 x 8192 168 -> 196). This warp uses one
// entry in nine, so it cannot wait on the entry's own `empty` barrier, whose
// parity would repeat in between: the MMA issuer commits the phase's entry 1,
// the previous user of the RoPE slice's place (kN = 3 entries before entry 4),
// to `free` as well, once per K phase.
template <bool PAIR, class Wait, class Full, class Arrive>
__device__ __forceinline__ void load_rope(const DecodeParams& p, const PieceIter& it, RowTable* rt, uint8_t* ring,
                                          uint64_t* free, int lane, int rank, Wait wait, Full full, Arrive arrive) {
  static_assert(kN == 3, "entry 4 takes the place of entry 1");
  const uint8_t* cache = static_cast<const uint8_t*>(p.kcache) + kFp4RopeOff + 16 * (lane & 7);
  Phases<PAIR> ph;
  ph.it = it;
  RingPos pos;
  while (ph.next()) {
    pos.advance(4);
    if (!ph.is_k()) continue;
    const int step = ph.step(), d = step % kRowDepth;
    if (!wait_warp(&rt->full[d], (step / kRowDepth) & 1, wait)) break;
    // rows first: nothing but the copies is left to do once the place is free
    const int32_t* rows = rt->row[d] + entry_token<PAIR>(true, 0, rank) + (lane >> 3);
    int row[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) row[i] = rows[4 * i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&rt->empty[d]);
    if (!wait_warp(free, step & 1, wait)) break;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      cp_async16(sw128(ring + pos.slot * kSlot, 4 * i + (lane >> 3), lane & 7),
                 cache + (size_t)(row[i] >= 0 ? row[i] : 0) * kFp4RecordBytes, row[i] >= 0 ? 16u : 0u);
    cp_async_mbar_arrive(full(pos.slot));
    __syncwarp();
    if (lane < 4) arrive(pos.slot, lane);
    pos.advance(1);
  }
  cp_async_wait_all();  // no copy may land after the CTA has finished, also where a wait above gave up
}

// ---------------------------------------------------------------- converters
// Group g of four warps converts latent entries g and g + 2 of every phase. A
// thread converts four items of 32 codes: tokens 32 w + 8 j + lane % 8, quarter
// lane / 8 of the entry's 128 dims; eight neighbouring lanes write the same
// chunk of eight rows, which the swizzle spreads over all banks. A group's
// entries are at most kN apart, so its waits on `empty` miss no phase. The raw bytes
// are taken into registers first, so that the next entry's copies overlap the
// conversion.
// Before the first entry of a piece all eight warps bring its query into form:
// by then the ring has made sure that the piece before is done with its own.
// wait(bar, parity): the kernel's bounded wait; arrive(slot, w): warp w of four has its part of the entry;
// query(piece): waits for the piece's query and brings this warp's rows into form.
template <bool PAIR, class Wait, class Arrive, class Query>
__device__ __forceinline__ void convert_ring(const PieceIter& it, RowTable* rt, uint8_t* ring, const uint8_t* raw,
                                             uint64_t* empty, int cw, int lane, Wait wait, Arrive arrive, Query query) {
  static_assert(kGroups == 2 && kRaw == 2, "each group has the raw buffer of its number");
  const int grp = cw >> 2, w = cw & 3;
  const int tok = 32 * w + (lane & 7), q = lane >> 3;
  const uint8_t* buf = raw + grp * kRawBytes;
  Phases<PAIR> ph;
  ph.it = it;
  RingPos pos;        // first entry of the phase
  uint32_t use = 0;   // uses of the raw buffer
  int piece = 0;
  bool stop = false;
  while (!stop && ph.next()) {
    if (ph.h == 0 && !query(piece++)) break;
#pragma unroll 1
    for (int e = grp; e < 4; e += 2, ++use) {
      const RingPos at = pos.at(e);
      if (!wait_warp(&rt->raw_full[grp], use & 1, wait)) { stop = true; break; }
      uint4 codes[4];
      uint32_t sc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        codes[j] = *reinterpret_cast<const uint4*>(buf + ((4 * w + j) * 32 + lane) * 16);
        sc[j] = *reinterpret_cast<const uint16_t*>(buf + 8192 + (tok + 8 * j) * 8 + 2 * q);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&rt->raw_empty[grp]);
      if (!wait_warp(&empty[at.slot], at.parity ^ 1u, wait)) { stop = true; break; }
      uint8_t* s = ring + at.slot * kSlot + (q >> 1) * kSlice;
#pragma unroll
      for (int j = 0; j < 4; ++j) store_item(codes[j], sc[j], s, tok + 8 * j, 4 * (q & 1));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive(at.slot, w);
    }
    pos.advance(ph.is_k() ? 5 : 4);
  }
}

}  // namespace fp4
}  // namespace mla
