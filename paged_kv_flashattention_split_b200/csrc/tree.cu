// tree.cu - attention of drafted tree nodes over the paged cache (bf16 or E4M3 pools), on the
// 5th-generation tensor cores.
//
// Node i of request r sees the p_r keys of the cached prefix, itself and its ancestors:
//     O_i = sum_j softmax_j(sm_scale q_i . K_j) V_j  over those keys,  lse_i = log sum_j exp(...).
// The rows of a query tile are the (node, query head) pairs of one KV head, 256 / G nodes a tile,
// so K and V are read once for all query heads and nodes that share them.
//
// One CTA per (slot of the plan's flat partition, KV head), 16 warps, one CTA per SM; it walks its
// slot's items (runs of 128-key tiles of one query tile):
//   warps 0-3      gather K (0, 1) and V (2, 3) rows slot by slot with 16-byte cp.async into rings in
//                  the tensor cores' 128-byte-swizzled layout: K by tiles of 128 keys, V by halves of
//                  64.  Filling a ring this way, and nothing else, measured 6.4-6.55 TB/s for pages of 8
//                  slots and more and 5.6 TB/s below, against 3.2-6.1 TB/s for one TMA box a page of 8 or
//                  16 slots and 6.8 TB/s at 64 and more, so one path serves every page size;
//   warp 4         issues the MMAs:  S_t = Q K^T,  O_t += P_t V  (M 128, N 128);
//   warps 6, 7     fetch the item's Q rows;
//   warps 8-15     two softmax warpgroups, one per stream t; thread = row.
// (E4M3 pools: 0-3 V, 5 and 6 K, 7 Q.)
// The two streams are the two 128-row halves of a query tile of more than 128 rows ("wide"), or,
// for fewer rows, the even and the odd key tiles of the same rows ("narrow"), so that in both the
// tensor cores work for one stream while the other is in its softmax.  TMEM, 512 columns: S_0, S_1,
// O_0, O_1.  P is written over S, 16 bits a value, and announced by halves of 64 keys, so PV of the
// lower half runs under the exponentials of the upper one.  All MMAs are issued by one thread and
// complete in order, so S complete implies that the PVs issued before it are.
//
// Softmax in one pass: a row's weights are 2^(score - ref) with a reference that is set by the first
// keys it sees and raised only when a score passes it by far, so nothing waits for a tile's maximum
// (8 requests of 128k tokens, 32 nodes, 64 heads, when it came in: 1.23 ms, against 1.38 with the maximum first).
//
// E4M3 pools.  K is used as it is: Q is split into two E4M3 terms whose sum is Q up to 2^-17 of its
// row's largest value (hi = round(q 2^e), lo = round(q 2^e - hi), a power of two a row, so every bf16
// range fits), and S = hi K^T + lo K^T takes two MMAs at twice the rate.  V is widened to f16 (exact)
// by the threads that fetched it, by bit operations: cvt shares its unit with ex2 (1650 clocks a tile).
//
// Visibility: only key tiles that reach past the prefix are masked, by the node's row of bits from
// the plan.  K/V rows of nodes that are not in use are not read at all (zeros in their place).
// Statistics are fp32.  P is rounded to bf16 (f16 for E4M3 pools) as the tensor cores need it; the
// row sum adds the unrounded values, so lse does not see that rounding.
//
// What bounds it (cold L2, plan and merge included; figures move with the box's clock).  64 requests of 512-8192
// tokens, up to 16 nodes, 32 / 8 heads: 218-240 us for 1.15 GB at page size 1, 210 where that takes 218 at page size
// 16: the copies, in pieces of 256 bytes, one KV head's row of a slot, by 144 of 148 SMs (loads alone 207-222).
// 8 x 128k tokens, 32 nodes, 64 / 8 heads: 1.14-1.34 ms for 4.3 GB and 1.1 PFLOP.  With all barriers in place the
// copies alone take 0.67 ms, the MMAs alone 0.82 (0.48 by 65 clocks each at 1965 MHz), the softmax alone 0.75, the
// barriers without work 0.56; the exponentials of two streams are 2320 clocks a key tile.  What is left is the chain
// of one stream's tile, S to P to PV to the next S, 4000 clocks, half of it covered by the other stream.  E4M3, up to
// 8 nodes: 0.19-0.2 ms for 0.58 GB, bound by the widening of V; wide trees are slower than in bf16, since one warp
// splits Q in front of every query tile (16 requests of 128-256 nodes, G 8, prefixes of 0-500 keys: 362 us, bf16 132).
// Tried and slower: S in steps of 64 keys with two buffers (an MMA of N 64 takes 49 clocks, of N 128
// 65); an issuing warp a stream (their MMAs interleave and both streams' scores come at once); four
// softmax warpgroups of half a key tile each; two regions of 64 score columns a stream, so that the next
// tile's scores are computed under this tile's exponentials (1.47 ms: the softmax never waits then, but the
// maximum has to come before the exponentials, and the two streams fall into step); chunks of 32 keys with the
// next one's scores on their way (1.45 ms); K and V released by the softmax warps, which saves the MMA warp
// two commits a turn (no change, E4M3 batch 6% slower); a quarter or more of the exponentials as polynomials on
// the FMA pipe; a register split by setmaxnreg (the E4M3 instance stopped with an illegal instruction;
// without the split all is well, so none is used).
//
// A piece that is a whole query tile is normalised and stored; otherwise its normalised O and its
// log-sum-exp go to the workspace, [32 groups of 4 d][256 rows] so that a warp's stores are whole
// lines, and tree_merge_kernel joins the pieces: lse = log2 sum 2^lse_s, O = sum 2^(lse_s - lse) O_s.
//
// Every wait on an mbarrier is bounded: on timeout the CTA records PA_ERR_DEVICE_INDEX in the
// workspace, every role stops, copies and MMAs in flight are drained and TMEM is freed.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "kernels.h"
#include "tma.cuh"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kHalf = 128 * 128;                 // bytes: 64 of the 128 d of 128 rows, 16 bits a value
constexpr int kTile = 2 * kHalf;                 // 32 KB: a Q tile, a K tile of bf16
constexpr int kVHalf = 64 * 128;                 // bytes: 64 of the 128 d of 64 rows, 16 bits a value
constexpr int kVUnit = 2 * kVHalf;               // 16 KB: V of 64 keys
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kWaitLimit = 1u << 20;
constexpr float kLn2 = 0.693147180559945309f;

// The rings, in flight or in use.  Three K tiles and four V halves; E4M3 pools keep their K tiles at
// 16 KB and have six more V halves, raw, a thread's pieces its own.  A bf16 tile's copies arrive on its
// barrier by themselves: with the copying warps announcing them after a wait, tiles that had landed
// were held back while a ring was full.
template <bool FP8> struct Cfg {
  static constexpr int kKRing = 3, kVRing = 4;
  static constexpr int kKTile = FP8 ? kTile / 2 : kTile;
  static constexpr int kLag = 2, kRaw = FP8 ? 2 * (kLag + 1) : 0;
  static constexpr int kKThreads = 64, kVThreads = 64, kQWarps = FP8 ? 1 : 2;
  // shared memory: barriers and small arrays first, then the tiles at the next 1024-byte border
  static constexpr int kBars = 2 * (kKRing + kVRing) + 14;
  static constexpr int kOffMl = 256;                                // float2 [2][128]: (max, sum) of both streams
  static constexpr int kOffExp = kOffMl + 2 * 128 * 8;              // int8 [2][256]: the Q rows' exponents (E4M3)
  static constexpr int kSmall = 3 * 1024;
  static constexpr int kOffQ = 0;                                   // from the tiles' base: two Q tiles
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kKRing * kKTile;
  static constexpr int kOffRaw = kOffV + kVRing * kVUnit;
  static constexpr int kTiles = kOffRaw + kRaw * (kVUnit / 2);
  static constexpr int kSmem = kSmall + kTiles;
  // P = 2^(x + kBias) with x a score's distance from the row's reference, which is raised when an x passes
  // kRaise.  bf16 has fp32's exponents: P <= 2^16, so sums over 2^17 keys of values up to 2^90 stay finite.
  // f16 keeps P between 2^-24 and 2^16: below 2^-14 it is off by up to 2^-25, and a row's sum is at least 2^6 (the
  // reference is less than 1 above the largest score it has seen), so a key's share by up to 2^-31.
  static constexpr float kBias = FP8 ? 7.f : 0.f, kRaise = FP8 ? 8.f : 16.f;
  // instruction descriptors: M 128, N 128, fp32 D; S: bf16 or E4M3, PV: bf16 or f16
  static constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | (FP8 ? 0u : (1u << 7) | (1u << 10));    // A (Q), B (K) K-major
  static constexpr uint32_t kIdescPV = kIdescS | (1u << 16);                           // B (V) MN-major
};
static_assert(Cfg<false>::kBars * 8 + 16 <= Cfg<false>::kOffMl && Cfg<false>::kOffExp + 512 <= Cfg<false>::kSmall &&
                  Cfg<false>::kSmem <= 232448 && Cfg<true>::kSmem <= 232448, "shared memory");

// ---------------------------------------------------------------- PTX helpers

// an arrival on `bar` (counted in its phase) once this thread's cp.async copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

// The MMA warp runs converged, with warp-uniform operands, and one elected lane's predicate on each
// tcgen05 instruction: operands then stay in uniform registers.  From inside an `if (lane == 0)` every
// operand of every MMA was moved there one by one: 85-110 clocks an MMA whatever its N.
//
// smem matrix descriptor: 128B swizzle, 8-row groups 1024 B apart (SBO), LBO as given; its low word is
// address / 16 + LBO / 16 * 2^16, its high word the constant below
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo_bytes) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) << 16);
}
// D (TMEM) (+)= A (shared memory) x B (shared memory), E4M3 or bf16
template <bool FP8>
__device__ __forceinline__ void tc_mma(uint32_t elected, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (FP8)
    asm volatile(
        "{\n.reg .pred p, e;\n.reg .b64 da, db;\nsetp.ne.b32 p, %5, 0;\nsetp.ne.b32 e, %0, 0;\n"
        "mov.b64 da, {%2, %6};\nmov.b64 db, {%3, %6};\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%1], da, db, %4, p;\n}\n"
        ::"r"(elected), "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p, e;\n.reg .b64 da, db;\nsetp.ne.b32 p, %5, 0;\nsetp.ne.b32 e, %0, 0;\n"
        "mov.b64 da, {%2, %6};\nmov.b64 db, {%3, %6};\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], da, db, %4, p;\n}\n"
        ::"r"(elected), "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
// D (TMEM) (+)= A (TMEM, K-major 16-bit pairs) x B (shared memory)
__device__ __forceinline__ void tc_mma_ts(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 db;\nsetp.ne.b32 p, %5, 0;\nsetp.ne.b32 e, %0, 0;\n"
      "mov.b64 db, {%3, %6};\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], db, %4, p;\n}\n"
      ::"r"(elected), "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.b32 e, %0, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}\n"
      ::"r"(elected), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// the same value in every lane, and known to be
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
        "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
        "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
        "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
        "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(uint64_t v, float* a, float* b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(*a), "=f"(*b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool FP8> __device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  return FP8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
// Two E4M3 codes, in the low bytes of the halves of x, to an f16 pair of 2^-8 times their values,
// exactly: a code's exponent and mantissa bits are those of an f16 whose exponent is 8 lower (its
// subnormals are f16 subnormals).  The factor 2^8 is in the launch's scales.  Bits instead of cvt,
// which shares its unit with ex2: 1650 clocks a tile of K or V by cvt.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  const uint32_t t = x * 128u;                   // sign at bit 14 of each half
  return t + (t & 0x40004000u);                  // moved to bit 15
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, 0, %2;\n" : "=r"(d) : "r"(a), "r"(sel));
  return d;
}
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t codes) {
  return make_uint2(e4m3x2_to_f16x2(prmt(codes, 0x4140u)), e4m3x2_to_f16x2(prmt(codes, 0x4342u)));
}

// One item of the plan: key tiles [k0, k1) of query tile t of request r.
struct Item {
  int r, L, prefix, row0, n, node0, rows, k0, k1;
  bool whole, shared_keys;                       // covers the query tile; other query tiles read the same keys
  __device__ __forceinline__ bool wide() const { return rows > 128; }
  __device__ __forceinline__ int nk() const { return k1 - k0; }
  // key tiles of stream t, and its i-th
  __device__ __forceinline__ int count(int t) const { return wide() ? nk() : (nk() + 1 - t) >> 1; }
  __device__ __forceinline__ int tile(int t, int i) const { return wide() ? i : 2 * i + t; }
};

__device__ __forceinline__ Item load_item(const TreeLaunch& a, int index) {
  const int4 it = a.ws.items[index];
  Item w;
  w.r = it.x;
  w.k0 = it.z;
  w.k1 = it.w;
  w.L = a.ws.req_len[it.x];
  w.prefix = a.ws.req_prefix[it.x];
  w.row0 = a.ws.req_aux[it.x];
  w.shared_keys = a.ws.req_splits[it.x] > 1;
  const int g = a.hq / a.hkv, qt = tree_tile_nodes(g);
  w.n = w.L - w.prefix;
  w.node0 = it.y * qt;
  w.rows = min(kTreeRows, (w.n - w.node0) * g);
  w.whole = w.k0 == 0 && w.k1 == (w.L + kTreeKvTile - 1) / kTreeKvTile;
  return w;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeLaunch a) {
  using C = Cfg<FP8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + C::kOffExp + 512 + 1023u) & ~1023u;   // the tiles
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t k_full = raw, k_empty = k_full + 8 * C::kKRing, v_full = k_empty + 8 * C::kKRing,
                 v_empty = v_full + 8 * C::kVRing, b0 = v_empty + 8 * C::kVRing;
  const uint32_t q_full = b0, q_empty = b0 + 8, o_done = b0 + 16, o_free = b0 + 24, ml_full = b0 + 32, drain = b0 + 40;
  auto s_full = [&](int t) -> uint32_t { return b0 + 48u + 8u * t; };
  auto p_full = [&](int t, int half) -> uint32_t { return b0 + 64u + 16u * t + 8u * half; };
  auto pv_lo = [&](int t) -> uint32_t { return b0 + 96u + 8u * t; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + 8 * C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + 8 * C::kBars + 8);
  float2* sm_ml = reinterpret_cast<float2*>(smem_raw + C::kOffMl);
  int8_t* sm_exp = reinterpret_cast<int8_t*>(smem_raw + C::kOffExp);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x / a.hkv, h_kv = blockIdx.x % a.hkv;
  // the merge (a programmatic dependent) may be scheduled; this grid waits for the one before it
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < C::kKRing; ++i) {
      mbar_init(k_full + 8u * i, C::kKThreads);                // the copying threads
      mbar_init(k_empty + 8u * i, 1);
    }
    for (int i = 0; i < C::kVRing; ++i) {
      if (i < C::kVRing / 2) mbar_init(v_full + 8u * i, 2 * C::kVThreads);   // a tile: both halves
      mbar_init(v_empty + 8u * i, 1);
    }
    mbar_init(q_full, C::kQWarps);
    mbar_init(q_empty, 1);
    mbar_init(o_done, 1);
    mbar_init(o_free, 8);                                      // the softmax warps
    mbar_init(ml_full, 8);
    mbar_init(drain, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(pv_lo(t), 1);                                  // PV of the lower half is done
      mbar_init(p_full(t, 0), 4);
      mbar_init(p_full(t, 1), 4);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  PlanHeader* hdr = a.ws.hdr;
  if (hdr->magic != kMagic || hdr->mode != PA_MODE_TREE || slot >= hdr->slots ||
      base + C::kTiles > raw + C::kSmem) {                     // (the last: a base of dynamic memory below 256-byte alignment)
    if (tid == 0 && blockIdx.x == 0) set_device_error(hdr, PA_ERR_WORKSPACE);
    return;
  }
  const int first = a.ws.slot_first[slot], last = min(a.ws.slot_first[slot + 1], hdr->num_items);
  if (first >= last) return;
  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
                 ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int g = a.hq / a.hkv, gshift = g == 1 ? 0 : g == 2 ? 1 : g == 4 ? 2 : 3;

  // bounded wait of a whole warp, with uniform control flow (a loop that lanes leave one by one costs twice
  // as much): false, and the CTA-wide abort flag set, if the barrier never completes
  auto wwait = [&](uint32_t b, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
      if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
      if (__any_sync(0xffffffffu, *abort_flag)) return false;
    }
    *abort_flag = 1;
    if (lane == 0) set_device_error(hdr, PA_ERR_DEVICE_INDEX);
    return false;
  };

  // until place u of a ring is free (u counts from the kernel's start)
  auto ring_free = [&](uint32_t bars, uint32_t u, uint32_t n) -> bool {
    return u < n || wwait(bars + 8u * (u % n), (u / n - 1) & 1u);
  };
  // The slot of key `key` of an item that ends before `end`, with table entry `page`: -1 (a row of zeros) past
  // the end and for a node that is not in use, flagged and -1 outside the pool.  32 bits do: num_slots < 2^31.
  const uint32_t last_page = (uint32_t)(a.num_slots - 1) >> a.page_shift, page_mask = (1u << a.page_shift) - 1u;
  auto slot_of_key = [&](const Item& w, int end, int key, int page) -> int {
    if (key >= end) return -1;
    const int x = key - w.prefix;
    if (x >= 0 && !((a.ws.tree_bits[(size_t)(w.row0 + x) * kTreeWords + (x >> 5)] >> (x & 31)) & 1u)) return -1;
    const uint32_t s = ((uint32_t)page << a.page_shift) | ((uint32_t)key & page_mask);
    if ((uint32_t)page > last_page || s >= (uint32_t)a.num_slots) {
      set_device_error(hdr, PA_ERR_DEVICE_INDEX);
      return -1;
    }
    return (int)s;
  };
  const uint32_t slot_bytes = (uint32_t)a.hkv * kHeadDim * (FP8 ? 1 : 2);
  auto row_of = [&](const char* pool, int s) { return pool + (uint64_t)(uint32_t)s * slot_bytes; };   // one 32 x 32 product

  const bool k_warp = FP8 ? warp == 5 || warp == 6 : warp < 2, v_warp = FP8 ? warp < 4 : warp == 2 || warp == 3;
  if (k_warp || (v_warp && !FP8)) {
    // ------------------------------------------------------------ copies of rows as they are
    // a step is 64 keys, 32 rows a warp, 16 lanes a row (8 for E4M3 K)
    constexpr int kRowLanes = FP8 ? 8 : 16, kPer = 32 / kRowLanes, kIters = 32 / kPer;
    const int wrow = FP8 ? 32 * (warp - 5) : 32 * (warp & 1);  // the warp's first row of a step
    const int sub = lane / kRowLanes, c16 = lane % kRowLanes;  // row of an instruction, 16-byte piece of the row
    const bool is_v = v_warp;
    const uint32_t half_bytes = is_v ? kVHalf : kHalf;         // from the first 64 d to the second
    const char* pool = static_cast<const char*>(is_v ? a.v_pool : a.k_pool) +
                       (size_t)h_kv * kHeadDim * (FP8 ? 1 : 2) + 16 * c16;
    // smem offsets of the thread's pieces: rows kPer i + sub; the swizzle repeats after 8 rows
    uint32_t off[8 / kPer];
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i)
      off[i] = (c16 >> 3) * half_bytes + (wrow + sub) * 128 + (((c16 & 7) ^ ((kPer * i + sub) & 7)) << 4);
    const uint64_t once = l2_evict_first();
    uint64_t keep;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(keep));
    uint32_t tiles = 0;                                        // key tiles of the items before
    bool ok = true;
#pragma unroll 1
    for (int index = first; ok && index < last; ++index) {
      const Item w = load_item(a, index);
      const uint64_t policy = w.shared_keys ? keep : once;
      const int n = 2 * w.nk(), key0 = w.k0 * kTreeKvTile + wrow + lane, end = min(w.L, w.k1 * kTreeKvTile);
      const int32_t* table = a.page_table + (size_t)w.r * a.pt_pitch;
      // the table entries as they are: they are read ahead, so nothing may depend on them at the load
      auto entry = [&](int key) -> int { return key < end ? __ldg(table + (key >> a.page_shift)) : 0; };
      int p0 = entry(key0), p1 = entry(key0 + 64), p2 = entry(key0 + 128);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int slots = slot_of_key(w, end, key0 + 64 * i, p0);
        p0 = p1;
        p1 = p2;
        p2 = entry(key0 + 64 * (i + 3));
        uint32_t dst, full;
        if (is_v) {
          const uint32_t u = 2 * tiles + i;
          if (!(ok = ring_free(v_empty, u, C::kVRing))) break;
          dst = base + C::kOffV + (u % C::kVRing) * kVUnit;
          full = v_full + 8u * ((u >> 1) % (C::kVRing / 2));
        } else {
          const uint32_t u = tiles + (i >> 1), place = u % C::kKRing;
          if (!(i & 1) && !(ok = ring_free(k_empty, u, C::kKRing))) break;
          dst = base + C::kOffK + place * C::kKTile + (i & 1) * (64 * 128);
          full = i & 1 ? k_full + 8u * place : 0u;
        }
        const bool whole = __all_sync(0xffffffffu, slots >= 0);
        int sl[kIters];                                        // all shuffles first: their latency is paid once
#pragma unroll
        for (int j = 0; j < kIters; ++j) sl[j] = __shfl_sync(0xffffffffu, slots, j * kPer + sub);
        if (whole) {
#pragma unroll
          for (int j = 0; j < kIters; ++j)
            cp_async_16_hint(dst + off[j % (8 / kPer)] + j * kPer * 128, row_of(pool, sl[j]), 16, policy);
        } else {
#pragma unroll
          for (int j = 0; j < kIters; ++j)
            cp_async_16_hint(dst + off[j % (8 / kPer)] + j * kPer * 128, row_of(pool, max(sl[j], 0)), sl[j] >= 0 ? 16 : 0,
                             policy);
        }
        if (full) cp_async_arrive(full);                       // when this thread's copies so far have landed
      }
      tiles += w.nk();
    }
    cp_async_wait<0>();
  } else if (v_warp) {
    // ------------------------------------------------------------ E4M3 V: fetched raw, widened to f16
    if constexpr (FP8) {
      // two warps a half of a key tile, 32 rows a warp, 8 lanes a row.  A lane's 16 codes are two 16-byte
      // pieces of f16; the lanes of the upper half of a row store the odd one first: eight lanes, eight pieces,
      // no bank twice.  Four rows on, the swizzle flips its bit 2.
      const int key_half = warp >> 1, wrow = 32 * (warp & 1), ptid = tid & 63;
      const int sub = lane >> 3, c16 = lane & 7, half = c16 >> 2, piece = (2 * c16) & 7;
      const char* pool = static_cast<const char*>(a.v_pool) + (size_t)h_kv * kHeadDim + 16 * c16;
      const uint32_t off_a = half * kVHalf + (wrow + sub) * 128 + (((piece + half) ^ sub) << 4);
      const uint32_t off_b = half * kVHalf + (wrow + sub) * 128 + (((piece + 1 - half) ^ sub) << 4);
      const uint64_t once = l2_evict_first();
      uint64_t keep;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(keep));
      uint32_t issued = 0, done = 0;                           // tiles of all items
      bool ok = true;
      auto raw_at = [&](uint32_t u) { return C::kOffRaw + (2 * (u % (C::kLag + 1)) + key_half) * (kVUnit / 2) + 16 * ptid; };
      auto widen = [&]() -> bool {                             // the oldest tile, whose copies by this thread have landed
        const uint32_t place = (2 * done + key_half) % C::kVRing;
        if (!ring_free(v_empty, 2 * done + key_half, C::kVRing)) return false;
        const uint8_t* src = base_ptr + raw_at(done);
        uint8_t* dst = base_ptr + C::kOffV + place * kVUnit;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // the eight codes of the piece that is stored first, then the others
          const uint2 xa = *reinterpret_cast<const uint2*>(src + i * 1024 + 8 * half);
          const uint2 xb = *reinterpret_cast<const uint2*>(src + i * 1024 + 8 * (1 - half));
          const uint2 a0 = e4m3x4_to_f16x4(xa.x), a1 = e4m3x4_to_f16x4(xa.y);
          const uint2 b0 = e4m3x4_to_f16x4(xb.x), b1 = e4m3x4_to_f16x4(xb.y);
          const uint32_t flip = (i & 1) << 6;
          *reinterpret_cast<uint4*>(dst + (off_a ^ flip) + i * 512) = make_uint4(a0.x, a0.y, a1.x, a1.y);
          *reinterpret_cast<uint4*>(dst + (off_b ^ flip) + i * 512) = make_uint4(b0.x, b0.y, b1.x, b1.y);
        }
        fence_proxy_async();
        mbar_arrive(v_full + 8u * (done % (C::kVRing / 2)));
        ++done;
        return true;
      };
#pragma unroll 1
      for (int index = first; ok && index < last; ++index) {
        const Item w = load_item(a, index);
        const uint64_t policy = w.shared_keys ? keep : once;
        const int n = w.nk(), key0 = w.k0 * kTreeKvTile + 64 * key_half + wrow + lane;
        const int end = min(w.L, w.k1 * kTreeKvTile);
        const int32_t* table = a.page_table + (size_t)w.r * a.pt_pitch;
        auto entry = [&](int key) -> int { return key < end ? __ldg(table + (key >> a.page_shift)) : 0; };
        int p0 = entry(key0), p1 = entry(key0 + kTreeKvTile);
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
          const int slots = slot_of_key(w, end, key0 + j * kTreeKvTile, p0);
          p0 = p1;
          p1 = entry(key0 + (j + 2) * kTreeKvTile);
          const uint32_t dst = base + raw_at(issued);
          int sl[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) sl[i] = __shfl_sync(0xffffffffu, slots, 4 * i + sub);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            cp_async_16_hint(dst + i * 1024, row_of(pool, max(sl[i], 0)), sl[i] >= 0 ? 16 : 0, policy);
          cp_async_commit();
          if (++issued > C::kLag) {
            cp_async_wait<C::kLag>();
            ok = widen();
          }
        }
      }
      cp_async_wait<0>();
#pragma unroll 1
      while (ok && done < issued) ok = widen();
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    // The streams take turns, PV of one key tile and then the scores of its next, so that they settle half
    // a period apart: one's MMAs run under the other's softmax.  (With a warp a stream their MMAs
    // interleaved, both streams' scores came at the same time, and softmax and MMAs alternated.)
    const uint32_t elected = elect_one();
    const uint32_t idesc_s = C::kIdescS | (a.negate ? 1u << 13 : 0u);      // S = -Q K^T for a negative scale
    const uint32_t tm = uniform(tmem);
    const uint32_t q_lo = uniform(desc_lo(base + C::kOffQ, 16));
    const uint32_t k_lo = uniform(desc_lo(base + C::kOffK, 16)), v_lo = uniform(desc_lo(base + C::kOffV, kVHalf));
    // K and V tiles are used in the order they are loaded, whichever stream's turn it is: their places in the
    // rings only move on
    constexpr uint32_t kVTiles = C::kVRing / 2;
    uint32_t ks = 0, k_par = 0, vs = 0, v_par = 0, items = 0, p_par = 0;   // bit t of p_par: the phase of stream t's P
    bool ok = true;
    // One item.  Wide: the streams share every K and V tile; narrow: they take them by turns.  The scores run
    // one key tile ahead of PV.
    auto run = [&](auto is_wide, int count0, int count1) -> bool {         // count0 >= count1
      constexpr bool kWide = decltype(is_wide)::value;
#pragma unroll 1
      for (int i = -1; i < count0; ++i) {
        // the item before has been read out of TMEM
        if (i == 0 && items > 0 && !wwait(o_free, (items - 1) & 1)) return false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int count = t ? count1 : count0;
          const bool pv = i >= 0 && i < count, scores = i + 1 < count;
          const bool fresh = !kWide || t == 0, last_use = !kWide || t == 1;   // of the K and V tiles
          // all that the turn reads is there before it waits for P: from P to the next scores nothing else is
          // waited for.  cp.async wrote it through the generic proxy, the MMAs read through the async one.
          if (fresh) {
            if (pv && !wwait(v_full + 8u * vs, v_par)) return false;
            if (scores && !wwait(k_full + 8u * ks, k_par)) return false;
            fence_proxy_async();
          }
          const uint32_t t_s = tm + 128 * t, t_o = tm + 256 + 128 * t;
          if (pv) {                                                        // O_t += P V, P from TMEM
            const uint32_t v0 = uniform(v_lo + vs * (2 * kVUnit >> 4)), acc = i > 0;
            if (!wwait(p_full(t, 0), (p_par >> t) & 1u)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ts(elected, t_o, t_s + 8 * kk, v0 + kk * (16 * 128 >> 4), C::kIdescPV, kk == 0 ? acc : 1u);
            tc_commit(elected, pv_lo(t));
            if (last_use) tc_commit(elected, v_empty + 16u * vs);
            if (!wwait(p_full(t, 1), (p_par >> t) & 1u)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ts(elected, t_o, t_s + 32 + 8 * kk, v0 + (kVUnit >> 4) + kk * (16 * 128 >> 4), C::kIdescPV, 1u);
            p_par ^= 1u << t;
          }
          if (scores) {
            const uint32_t kb = uniform(k_lo + ks * (C::kKTile >> 4));
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              // bf16: 16 d a step, 64 d a half; E4M3: 32 d a step, first of the high, then of the low terms
              const uint32_t q_off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
              const uint32_t k_off = FP8 ? ((kk & 3) * 32) >> 4 : q_off;
              tc_mma<FP8>(elected, t_s, q_lo + (kWide ? t : 0) * (kTile >> 4) + q_off, kb + k_off, idesc_s, kk > 0);
            }
            tc_commit(elected, s_full(t));
            if (last_use) tc_commit(elected, k_empty + 8u * ks);
          }
          if (pv && last_use) {
            tc_commit(elected, v_empty + 16u * vs + 8u);
            vs = vs + 1 == kVTiles ? 0 : vs + 1;
            v_par ^= vs == 0;
          }
          if (scores && last_use) {
            ks = ks + 1 == C::kKRing ? 0 : ks + 1;
            k_par ^= ks == 0;
          }
        }
        if (i + 2 == count0) tc_commit(elected, q_empty);
      }
      return true;
    };
#pragma unroll 1
    for (int index = first; ok && index < last; ++index, ++items) {
      const Item w = load_item(a, index);
      const int count0 = uniform(w.count(0)), count1 = uniform(w.count(1));
      if (!(ok = wwait(q_full, items & 1))) break;
      ok = uniform(w.wide()) ? run(std::true_type(), count0, count1) : run(std::false_type(), count0, count1);
      if (ok) tc_commit(elected, o_done);
    }
    // all issued tensor-core work has finished before TMEM is released
    tc_commit(elected, drain);
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit && !__all_sync(0xffffffffu, mbar_try_wait(drain, 0)); ++i) {}
    __syncwarp();
  } else if (warp == 5) {
    // bf16 pools: nothing to do
  } else if (warp < 8) {
    // ------------------------------------------------------------ Q rows
    const int q_warp = FP8 ? 0 : warp - 6;
    uint32_t items = 0;
#pragma unroll 1
    for (int index = first; index < last; ++index, ++items) {
      const Item w = load_item(a, index);
      if (items > 0 && !wwait(q_empty, (items - 1) & 1)) break;
      const int c = lane & 15;
      // row: (node, query head of the group); rows past the item's stay as they are (their results are not used)
      const uint16_t* q0 = a.q + ((size_t)(w.row0 + w.node0) * a.hq + (size_t)h_kv * g) * kHeadDim + 8 * c;
      // 16-byte unit u of a row's half h
      auto at = [&](int row, int h, int u) -> uint32_t {
        return C::kOffQ + (row >> 7) * kTile + h * kHalf + (row & 127) * 128 + ((u ^ (row & 7)) << 4);
      };
#pragma unroll 4
      for (int row = 2 * q_warp + (lane >> 4); row < w.rows; row += 2 * C::kQWarps)
        cp_async_16(base + at(row, c >> 3, c & 7), q0 + ((size_t)(row >> gshift) * a.hq + (row & (g - 1))) * kHeadDim, 16);
      cp_async_commit();
      cp_async_wait<0>();
      if constexpr (FP8) {
        // In place: a bf16 row's two halves of 128 bytes become its high and low E4M3 terms.  With the row's
        // largest value in [2^7, 2^8), a value down to 2^-9 of it is hi + lo exactly (8 significant bits in
        // 4 + 4); below, lo's step is 2^-9, so q 2^e is off by at most 2^-10.
#pragma unroll 2
        for (int row0 = 0; row0 < w.rows; row0 += 2) {
          const int row = row0 + (lane >> 4);
          const bool live = row < w.rows;
          const uint4 v = *reinterpret_cast<const uint4*>(base_ptr + at(live ? row : row0, c >> 3, c & 7));
          const uint32_t word[4] = {v.x, v.y, v.z, v.w};
          float f[8], mx = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo_to_f32(word[i]);
            f[2 * i + 1] = bf16hi_to_f32(word[i]);
            mx = fmaxf(mx, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
          }
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int e = max(-119, min(127, (int)(__float_as_uint(mx) >> 23) - 127));   // 2^e <= mx, above 2^-119
          const float up = mx < __int_as_float(0x7f800000) ? __int_as_float((127 + 7 - e) << 23) : __int_as_float(0x7fc00000);
          uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = make_float2(f[2 * i] * up, f[2 * i + 1] * up);
            const __nv_fp8x2_storage_t h8 = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(h8, __NV_E4M3);
            const float2 back = make_float2(__half2float(__ushort_as_half(hr.x)), __half2float(__ushort_as_half(hr.y)));
            const __nv_fp8x2_storage_t l8 =
                __nv_cvt_float2_to_fp8x2(make_float2(x.x - back.x, x.y - back.y), __NV_SATFINITE, __NV_E4M3);
            hi[i >> 1] |= (uint32_t)h8 << (16 * (i & 1));
            lo[i >> 1] |= (uint32_t)l8 << (16 * (i & 1));
          }
          __syncwarp();                                        // the rows have been read
          if (live) {
            *reinterpret_cast<uint2*>(base_ptr + at(row, 0, c >> 1) + 8 * (c & 1)) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(base_ptr + at(row, 1, c >> 1) + 8 * (c & 1)) = make_uint2(lo[0], lo[1]);
            if (c == 0) sm_exp[(items & 1) * 256 + row] = (int8_t)(e - 7);
          }
          __syncwarp();
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int t = (warp - 8) >> 2;                             // stream
    const int lrow = 32 * (warp & 3) + lane;                   // TMEM lane
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + 128 * t + lane_off, t_o = tmem + 256 + lane_off;
    const float NEG_INF = -__int_as_float(0x7f800000);
    uint32_t s_par = 0, ml_par = 0, items = 0;
    bool ok = true;
#pragma unroll 1
    for (int index = first; ok && index < last; ++index, ++items) {
      // what the loop over the key tiles needs of the item; the rest is read again behind it, so that no
      // registers are held meanwhile
      bool live_warp, in_use = false;                          // some row of this warp is in the tile; this row is a node in use
      int count, node_of_key, key_step, bits_row, exp_row;              // node_of_key: < 0 in the prefix
      {
        const Item w = load_item(a, index);
        const int row = lrow + (w.wide() ? 128 * t : 0);
        live_warp = (row & ~31) < w.rows;
        count = w.count(t);
        node_of_key = (w.k0 + w.tile(t, 0)) * kTreeKvTile - w.prefix;
        key_step = w.wide() ? kTreeKvTile : 2 * kTreeKvTile;
        exp_row = min(row, w.rows - 1);
        const int node = w.node0 + (row >> gshift);
        bits_row = w.row0 + min(node, w.n - 1);
        if (row < w.rows) in_use = (a.ws.tree_bits[(size_t)bits_row * kTreeWords + (node >> 5)] >> (node & 31)) & 1u;
      }
      // The row's reference (a whole number; the weights are 2^(score - ref)) and sum
      float ref = 0.f, l = 0.f;
      float limit;                                             // what raises it: never for a row of no use, whatever it holds
      limit = in_use ? NEG_INF : -NEG_INF;
      float c = a.scale_log2;
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        if (!(ok = wwait(s_full(t), s_par))) break;
        s_par ^= 1u;                                           // also the phase after this tile's pv_lo
        tc_fence_after();
        if (!live_warp) {                                      // no rows: keep the barriers going
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(p_full(t, 0));
            mbar_arrive(p_full(t, 1));
          }
          continue;
        }
        if (FP8 && i == 0) {
          const int e = sm_exp[(items & 1) * 256 + exp_row];
          c = fmaxf(a.scale_log2 * __int_as_float((127 + e) << 23), 1e-37f);
        }
        // An item's first half, where all rows see all of it, sets the references without a second pass over it.
        if (i == 0 && node_of_key <= -64) {
          float top[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
          uint32_t v[64];
          __syncwarp();
          tmem_ld64(t_s, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) top[e & 3] = max3(top[e & 3], __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          const float most = c * fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          if (in_use && most > NEG_INF) {
            ref = ceilf(most);
            limit = C::kRaise + C::kBias;
          }
        }
        // One pass over halves of 64 keys: no maximum of the tile is taken before its exponentials.  A row
        // keeps its reference until some score passes it by 2^kRaise (or, the first time, until it sees a
        // key); then, before this half's P is stored, the reference rises to the half's maximum, O and the
        // sum are scaled down and the half is taken again.  (Nothing of the half is held over that: the
        // registers it would cost made the usual path slower, 1.74 instead of 1.11 ms for 8 x 128k tokens.)
#pragma unroll 1
        for (int step = 0; step < 4; ++step) {                 // even: the half; odd: the half again, if a row was raised
          const int half = step >> 1;
          uint32_t v[64];
          __syncwarp();
          tmem_ld64(t_s + 64 * half, v);
          const int x0 = node_of_key + i * key_step + 64 * half;   // node at the half's first key
          if (x0 > -64) {
            // bit e of a mask: the half's key (32 +) e is in the prefix, the node itself or an ancestor
            const uint32_t* bits = a.ws.tree_bits + (size_t)bits_row * kTreeWords;
            uint32_t mask[2];
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const int x = x0 + 32 * cc;
              if (x <= -32) mask[cc] = 0xffffffffu;
              else if (x < 0) mask[cc] = (bits[0] << -x) | ((1u << -x) - 1u);
              else {
                const uint32_t lo = x < 256 ? bits[x >> 5] : 0u, hi = x < 224 ? bits[(x >> 5) + 1] : 0u;
                mask[cc] = __funnelshift_r(lo, hi, x & 31);
              }
            }
            __syncwarp();
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!((mask[e >> 5] >> (e & 31)) & 1u)) v[e] = __float_as_uint(NEG_INF);
          } else {
            tmem_wait_ld();
          }
          // the distances from the reference (plus kBias), and the largest
          const uint64_t c2 = f32x2(c, c), r2 = f32x2(C::kBias - ref, C::kBias - ref);
          float top[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float y0, y1;
            split2(fma2(f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, r2), &y0, &y1);
            top[e & 3] = max3(top[e & 3], y0, y1);
            v[2 * e] = __float_as_uint(y0);
            v[2 * e + 1] = __float_as_uint(y1);
          }
          // P, before it is known whether a row is raised: the exponentials need not wait for the maximum
          uint64_t sum[2] = {0, 0};
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ex2(__uint_as_float(v[2 * e])), p1 = ex2(__uint_as_float(v[2 * e + 1]));
            sum[e & 1] = add2(sum[e & 1], f32x2(p0, p1));
            pk[e] = pack_p<FP8>(p0, p1);
          }
          const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          const bool raise = most > limit;
          if (!(step & 1) && __any_sync(0xffffffffu, raise)) {
            const float up = raise ? ceilf(most - C::kBias) : 0.f;
            const float alpha = raise && limit != NEG_INF ? ex2(-up) : 1.f;   // the first time l and O are 0 (or O is not there)
            ref += up;
            if (raise) limit = C::kRaise + C::kBias;
            l *= alpha;
            if (__any_sync(0xffffffffu, alpha != 1.f) && i + half > 0) {
              // O_t is stable: S_t complete implies PV_t of the tile before, and PV of the lower half, which
              // has been announced, is waited for
              if (half && !(ok = wwait(pv_lo(t), s_par ^ 1u))) break;
              tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < kHeadDim; d += 16) {         // 16 at a time: registers
                uint32_t ov[16];
                tmem_ld16(t_o + 128 * t + d, ov);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                tmem_st16(t_o + 128 * t + d, ov);
              }
              tmem_wait_st();
            }
            continue;
          }
          tmem_st32(t_s + 32 * half, pk);                      // over scores that have been read
          float s0, s1;
          split2(add2(sum[0], sum[1]), &s0, &s1);
          l += s0 + s1;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(t, half));
          step |= 1;
        }
        if (!ok) break;
      }
      const float m = limit == C::kRaise + C::kBias ? ref : NEG_INF;   // raised at all
      const Item w = load_item(a, index);
      const bool wide = w.wide();
      const int row = lrow + (wide ? 128 * t : 0);             // row of the query tile
      const int node = w.node0 + (row >> gshift);
      const bool used = in_use;
      if (!ok || !(ok = wwait(o_done, items & 1))) break;
      tc_fence_after();
      // wide: the row's 128 d from its own stream; narrow: 64 d of both streams' O, joined
      float f0 = 0.f, f1 = 0.f, lse2 = NEG_INF;                // factors of O_0, O_1 (wide: f0 of O_t)
      if (wide) {
        if (used && l > 0.f) {
          f0 = a.v_scale / l;
          lse2 = m + __log2f(l) - C::kBias;
        }
      } else {
        sm_ml[128 * t + lrow] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (!(ok = wwait(ml_full, ml_par))) break;
        ml_par ^= 1;
        const float2 x = sm_ml[lrow], y = sm_ml[128 + lrow];
        const float M = fmaxf(x.x, y.x);
        if (used && M != NEG_INF) {
          const float e0 = ex2(x.x - M), e1 = ex2(y.x - M), sum = x.y * e0 + y.y * e1;
          if (sum > 0.f) {
            f0 = e0 * a.v_scale / sum;
            f1 = e1 * a.v_scale / sum;
            lse2 = M + __log2f(sum) - C::kBias;
          }
        }
      }
      if (live_warp) {
        const bool two = !wide && w.nk() > 1;                  // O_1 holds something
        const int d_begin = wide ? 0 : 64 * t, d_end = wide ? 128 : 64 * t + 64;
        const size_t out_row = (size_t)(w.row0 + node) * a.hq + (size_t)h_kv * g + (row & (g - 1));
        // a piece that continues the slot before: 2 slot, one that the next slot continues: 2 slot + 1
        const size_t piece = (size_t)(2 * slot + (w.k0 == 0 ? 1 : 0)) * a.hkv + h_kv;
#pragma unroll 1
        for (int d = d_begin; d < d_end; d += 16) {            // by 32 the loop over the key tiles had spills
          uint32_t ov[16], ow[16];
          __syncwarp();                                        // the lanes of a warp read TMEM together
          tmem_ld16(t_o + (wide ? 128 * t : 0) + d, ov);
          if (two) tmem_ld16(t_o + 128 + d, ow);
          tmem_wait_ld();
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            o[e] = f0 != 0.f ? __uint_as_float(ov[e]) * f0 : 0.f;
            if (two && f1 != 0.f) o[e] = fmaf(__uint_as_float(ow[e]), f1, o[e]);
          }
          if (d + 16 >= d_end) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
          }
          if (row < w.rows && w.whole) {
            uint16_t* dst = a.out + out_row * kHeadDim + d;
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                                                              pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
          } else if (row < w.rows) {
            float4* dst = reinterpret_cast<float4*>(a.ws.partial_o) + (piece * 32 + d / 4) * kTreeRows + row;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[(size_t)e * kTreeRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (row < w.rows && (wide || t == 0)) {
          if (!w.whole) a.ws.partial_lse[piece * kTreeRows + row] = lse2;
          else if (a.lse_out) a.lse_out[out_row] = lse2 * kLn2;
        }
      } else if (lane == 0) {
        mbar_arrive(o_free);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// One CTA per (cut query tile, KV head, 32 rows): joins the tile's pieces.  A thread owns one row and 8
// of its d; the pieces' log-sum-exps are read by all warps at once for the maximum, then eight pieces'
// loads are in flight.
constexpr int kMergeThreads = 512;
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeLaunch a) {
  __shared__ float sm_max[kMergeThreads / 32][32];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  // the next layer's attention may be scheduled: it waits for this grid
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const PlanHeader* hdr = a.ws.hdr;
  if (hdr->magic != kMagic || hdr->mode != PA_MODE_TREE || (int)blockIdx.x >= hdr->reserved1) return;
  const int2 tile = a.ws.tree_tiles[blockIdx.x];
  const int g = a.hq / a.hkv, qt = tree_tile_nodes(g), h_kv = blockIdx.y;
  const int L = a.ws.req_len[tile.x], n = L - a.ws.req_prefix[tile.x], node0 = tile.y * qt;
  const int rows = min(kTreeRows, (n - node0) * g);
  if (32 * (int)blockIdx.z >= rows) return;
  const int ktiles = (L + kTreeKvTile - 1) / kTreeKvTile;
  const int u0 = a.ws.req_base[tile.x] + tile.y * ktiles, per = hdr->chunk_tiles;
  const int c0 = u0 / per, c1 = min((u0 + ktiles - 1) / per, a.slots - 1);
  const int lane = threadIdx.x & 31, dg = threadIdx.x >> 5;    // 16 warps: 8 d each
  const int row = 32 * blockIdx.z + lane;                      // rows of a piece behind the tile's hold anything
  // the piece of slot c: 2 c0 + 1 where the tile begins, 2 c where it goes on
  auto piece = [&](int c) -> size_t { return (size_t)(2 * c + (c == c0 ? 1 : 0)) * a.hkv + h_kv; };
  const float NEG_INF = -__int_as_float(0x7f800000);
  float M = NEG_INF;
  for (int c = c0 + dg; c <= c1; c += kMergeThreads / 32) M = fmaxf(M, a.ws.partial_lse[piece(c) * kTreeRows + row]);
  sm_max[dg][lane] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) M = fmaxf(M, sm_max[w][lane]);
  if (row >= rows) return;
  float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
  float sum = 0.f;
  if (M != NEG_INF) {
    const float4* po = reinterpret_cast<const float4*>(a.ws.partial_o);
#pragma unroll 8
    for (int c = c0; c <= c1; ++c) {
      const size_t p = piece(c);
      const float4 x = po[(p * 32 + 2 * dg) * kTreeRows + row], y = po[(p * 32 + 2 * dg + 1) * kTreeRows + row];
      const float f = ex2(a.ws.partial_lse[p * kTreeRows + row] - M);
      sum += f;
      lo = make_float4(fmaf(x.x, f, lo.x), fmaf(x.y, f, lo.y), fmaf(x.z, f, lo.z), fmaf(x.w, f, lo.w));
      hi = make_float4(fmaf(y.x, f, hi.x), fmaf(y.y, f, hi.y), fmaf(y.z, f, hi.z), fmaf(y.w, f, hi.w));
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const size_t out_row = (size_t)(a.ws.req_aux[tile.x] + node0 + row / g) * a.hq + (size_t)h_kv * g + row % g;
  *reinterpret_cast<uint4*>(a.out + out_row * kHeadDim + 8 * dg) =
      make_uint4(pack_bf16x2(lo.x * inv, lo.y * inv), pack_bf16x2(lo.z * inv, lo.w * inv),
                 pack_bf16x2(hi.x * inv, hi.y * inv), pack_bf16x2(hi.z * inv, hi.w * inv));
  if (dg == 0 && a.lse_out) a.lse_out[out_row] = M == NEG_INF ? NEG_INF : (M + __log2f(sum)) * kLn2;
}

template <bool FP8>
cudaError_t launch_tree_t(const TreeLaunch& a, cudaStream_t s) {
  static std::atomic<bool> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(tree_kernel<FP8>, Cfg<FP8>::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(tree_kernel<FP8>, dim3(a.slots * a.hkv), dim3(kThreads), Cfg<FP8>::kSmem, a, s);
  if (e != cudaSuccess) return e;
  return launch_programmatic(tree_merge_kernel, dim3(a.max_cut, a.hkv, kTreeRows / 32), dim3(kMergeThreads), 0, a, s);
}

}  // namespace

cudaError_t launch_tree(const TreeLaunch& a, cudaStream_t s) {
  return a.fp8 ? launch_tree_t<true>(a, s) : launch_tree_t<false>(a, s);
}

}  // namespace pa
