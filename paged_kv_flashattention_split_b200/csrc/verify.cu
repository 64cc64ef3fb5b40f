// verify.cu - verification of a tree of drafted tokens against the target's probabilities.
//
// The walk starts at node 0 (the last accepted token) and asks the children of the current node
// in index order.  With w the weights of the current node's target row (Z = 1 at first), q the
// draft row its children were drawn from and u the child's random number, child c of token x is
//     accepted  iff  u q(x) Z < w(x);    else  w <- max(w - Z q, 0),  Z <- sum w.
// Without draft rows the children are taken as given, q = the one-hot of x: w(x) <- 0,
// Z <- Z - w(x).  Where no child is accepted the next token is the smallest x with
//     w(0) + .. + w(x) > u_final * sum w,
// so accepted tokens and the next one together are distributed as the target's own samples.
//
// After k rejections at a node, w = max(p - c q, 0) with c = 1 + Z_1 + .. + Z_(k-1): subtractions that
// stop at zero add up, so a pass evaluates one product a token however many children were rejected.
//
// A cluster of CTAs serves one request.  Rank 0 reads the nodes, each with its two probabilities at
// its parent's rows, the other ranks copy them from its shared memory, and all ranks walk: they have
// the same numbers, so they take the same steps, and accepting costs no pass over the vocabulary.  A
// pass (a rejection with draft rows, or the final sum) is split over the cluster's CTAs: warps sum
// chunks of 512 weights, each CTA keeps its chunks' sums and sends its total to every rank, and one
// cluster barrier later every rank has the sum.  The final token is found by the CTA whose part
// holds it: from the totals, its chunk sums, then one chunk read again.
// What bounds it is the chain of passes of the request with the most rejections, each a read of its
// rows (from L2 after the first).  64 requests, trees of 8-32 nodes over 128k tokens: 47-52 us, of which
// the first pass, from HBM, is 10 (rows kept in shared memory between the passes: 56); 16 requests without draft
// rows, 64 nodes: 14 us; one chain of 8: 12 us.
//
// All weights and sums are 64-bit: a cumulative sum over 10^5 tokens in 32 bits is off by more
// than the gaps between neighbouring tokens' intervals.  The sums' order is fixed, so results
// repeat exactly.
#include <cooperative_groups.h>

#include "kernels.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 512;                      // tokens one warp sums at a time
constexpr int kQuads = kChunk / 128;             // float4 loads of a lane
constexpr int kMaxChunks = kVerifyMaxVocab / kChunk;
constexpr int kMaxCluster = 8;
constexpr int kNodes = kTreeMaxNodes;

struct Shared {
  double chunk_sum[kMaxChunks];
  double cta_sum[2][kMaxCluster];                // the CTAs' totals of a pass, by turns
  int32_t gone[kNodes];                          // without draft rows: rejected tokens of the current node
  int32_t parent[kNodes], token[kNodes];
  float u[kNodes], p[kNodes], q[kNodes];         // random number; target and draft value at the parent's row
  float u_final;
  int row0, n;
  // warp 0's decision: the pass to run, or the end
  double c;                                      // the weights are max(p - c q, 0)
  double threshold, before;                      // the end: u_final * sum, and the sum of the CTAs before the owner
  int done, row, rejected, owner;                // owner -1: there is no token to find
};

__device__ __forceinline__ double positive(float p) { return p > 0.f ? (double)p : 0.0; }   // a NaN counts as 0

// A probability as a double, exactly (one below the normal range, 2^-126, as 0, and so is -0): the fields moved
// by integer operations, beside the conversions of the other row, which run at a quarter of their rate.
__device__ __forceinline__ double by_bits(float q) {
  const uint32_t b = __float_as_uint(q);
  return __hiloint2double((int)b >= 0x00800000 ? (int)((b >> 3) + ((1023u - 127u) << 20)) : 0, (int)(b << 29));
}

// The weights of the current node's row, taken through the rejections so far.
struct Row {
  const float* p;
  const float* q;                                // NULL: one-hot drafts
  const int32_t* gone;
  double c;
  int rejected, vocab;
  bool wide;                                     // rows 16-byte aligned

  __device__ __forceinline__ float4 load(const float* row, int x) const {
    if (wide && x + 4 <= vocab) return __ldg(reinterpret_cast<const float4*>(row + x));
    float4 v;
    v.x = x < vocab ? row[x] : 0.f;
    v.y = x + 1 < vocab ? row[x + 1] : 0.f;
    v.z = x + 2 < vocab ? row[x + 2] : 0.f;
    v.w = x + 3 < vocab ? row[x + 3] : 0.f;
    return v;
  }
  __device__ __forceinline__ double weight(float p_x, float q_x) const {
    return fmax(fma(-c, by_bits(q_x), positive(p_x)), 0.0);
  }
  // the lane's 4 weights of step `it` of a chunk (tokens 128 it + 4 lane ..); dropped: its tokens gone, bit 4 it + e
  __device__ __forceinline__ void weights(int it, float4 vp, float4 vq, uint32_t dropped, double (&w)[4]) const {
    if (q && c > 0.0) {
      w[0] = weight(vp.x, vq.x);
      w[1] = weight(vp.y, vq.y);
      w[2] = weight(vp.z, vq.z);
      w[3] = weight(vp.w, vq.w);
      return;
    }
    w[0] = positive(vp.x);
    w[1] = positive(vp.y);
    w[2] = positive(vp.z);
    w[3] = positive(vp.w);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((dropped >> (4 * it + e)) & 1u) w[e] = 0.0;
  }
  // which of the lane's tokens of a chunk were rejected (one-hot drafts)
  __device__ __forceinline__ uint32_t dropped(int chunk, int lane) const {
    uint32_t bits = 0;
    if (q) return bits;
    for (int k0 = 0; k0 < rejected; k0 += 32) {
      const int x = k0 + lane < rejected ? gone[k0 + lane] - chunk * kChunk : -1;
      for (unsigned here = __ballot_sync(0xffffffffu, x >= 0 && x < kChunk); here; here &= here - 1) {
        const int at = __shfl_sync(0xffffffffu, x, __ffs(here) - 1);
        if (((at & 127) >> 2) == lane) bits |= 1u << (4 * (at >> 7) + (at & 3));
      }
    }
    return bits;
  }
  // the chunk's values, all loads in flight at once
  __device__ __forceinline__ void fetch(int chunk, int lane, float4 (&vp)[kQuads], float4 (&vq)[kQuads]) const {
#pragma unroll
    for (int it = 0; it < kQuads; ++it) {
      const int x = chunk * kChunk + it * 128 + 4 * lane;
      vp[it] = load(p, x);
      vq[it] = q && c > 0.0 ? load(q, x) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ double warp_scan(double x, int lane) {       // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ double chunk_total(const Row& row, int chunk, int lane) {
  const uint32_t dropped = row.dropped(chunk, lane);
  float4 vp[kQuads], vq[kQuads];
  row.fetch(chunk, lane, vp, vq);
  double sum = 0.0;
#pragma unroll
  for (int it = 0; it < kQuads; ++it) {
    double w[4];
    row.weights(it, vp[it], vq[it], dropped, w);
    sum += (w[0] + w[1]) + (w[2] + w[3]);
  }
  return warp_sum(sum);
}

// First token of the chunk with a positive weight whose cumulative sum passes the threshold; if
// rounding leaves none, the chunk's last token with a positive weight (-1: it has none).
__device__ int find_in_chunk(const Row& row, int chunk, double before, double threshold, int lane) {
  const uint32_t dropped = row.dropped(chunk, lane);
  float4 vp[kQuads], vq[kQuads];
  row.fetch(chunk, lane, vp, vq);
  int last = -1;
#pragma unroll
  for (int it = 0; it < kQuads; ++it) {
    const int x = chunk * kChunk + it * 128 + 4 * lane;
    double w[4];
    row.weights(it, vp[it], vq[it], dropped, w);
    const double sum = (w[0] + w[1]) + (w[2] + w[3]);
    const double incl = warp_scan(sum, lane);
    double cum = before + (incl - sum);
    int found = -1, mine = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cum += w[e];
      if (w[e] > 0.0) {
        mine = x + e;
        if (found < 0 && cum > threshold) found = x + e;
      }
    }
    const unsigned who = __ballot_sync(0xffffffffu, found >= 0);
    if (who) return __shfl_sync(0xffffffffu, found, __ffs(who) - 1);
    const unsigned any = __ballot_sync(0xffffffffu, mine >= 0);
    if (any) last = __shfl_sync(0xffffffffu, mine, 31 - __clz(any));
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return last;
}

__global__ void __launch_bounds__(kThreads, 2) verify_kernel(VerifyLaunch a) {
  __shared__ Shared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_chunks = (a.vocab + kChunk - 1) / kChunk;
  const int per = (n_chunks + ctas - 1) / ctas;
  const int c0 = min(n_chunks, rank * per), c1 = min(n_chunks, c0 + per);

  if (rank == 0) {
    const int row0 = a.cu_seqlens_q[r];
    const long long row1 = a.cu_seqlens_q[r + 1], cnt = row1 - row0;
    int n = (int)cnt;
    if (row0 < 0 || row1 > a.rows || cnt < 0 || cnt > kNodes) {
      if (tid == 0 && a.hdr) set_device_error(a.hdr, PA_ERR_DEVICE_INDEX);
      n = 0;
    }
    for (int i = tid; i < n; i += kThreads) {
      const int parent = a.parent[row0 + i], token = a.tokens[row0 + i];
      const bool bad = parent < -2 || parent >= i || (i > 0 && parent >= 0 && (token < 0 || token >= a.vocab));
      if (bad && a.hdr) set_device_error(a.hdr, PA_ERR_DEVICE_INDEX);
      const bool asks = i > 0 && parent >= 0 && !bad;
      sm.parent[i] = bad ? -2 : parent;
      sm.token[i] = token;
      sm.u[i] = asks ? a.u_accept[row0 + i] : 0.f;
      sm.p[i] = asks ? a.target[(size_t)(row0 + parent) * a.target_pitch + token] : 0.f;
      sm.q[i] = asks && a.draft ? a.draft[(size_t)(row0 + parent) * a.draft_pitch + token] : 1.f;
    }
    for (int64_t k = tid; k < a.path_pitch; k += kThreads) a.path[r * a.path_pitch + k] = -1;
    if (tid == 0) {
      sm.row0 = row0;
      sm.u_final = a.u_final[r];
    }
    __syncthreads();
    if (tid == 0) sm.n = n > 0 && sm.parent[0] == -1 ? n : 0;   // an idle request: its root is not in use
  }
  cluster.sync();                                // the nodes are there
  if (rank > 0) {
    const Shared* head = cluster.map_shared_rank(&sm, 0);
    const int n = head->n;
    for (int i = tid; i < n; i += kThreads) {
      sm.parent[i] = head->parent[i];
      sm.token[i] = head->token[i];
      sm.u[i] = head->u[i];
      sm.p[i] = head->p[i];
      sm.q[i] = head->q[i];
    }
    if (tid == 0) {
      sm.n = n;
      sm.row0 = head->row0;
      sm.u_final = head->u_final;
    }
  }
  __syncthreads();
  const int n = sm.n;
  if (n == 0) {
    if (rank == 0 && tid == 0) {
      a.accept_len[r] = 0;
      a.next_token[r] = -1;
    }
    cluster.sync();                              // rank 0's shared memory outlives its readers
    return;
  }

  // warp 0: the walk's state, the same in every lane
  int cur = 0, at = 1, taken = 0, rejected = 0;
  double Z = 1.0, c = 0.0;
  bool summed = false;                           // Z is the sum of w over the row (of the last pass)
  // runs the walk until a pass is needed (true) or it ends (false)
  auto walk = [&]() -> bool {
    while (at < n && taken + 1 < a.path_pitch) {
      // the next child of the current node, 32 nodes at a time
      const unsigned kids = __ballot_sync(0xffffffffu, at + lane < n && sm.parent[min(at + lane, n - 1)] == cur);
      if (!kids) {
        at += 32;
        continue;
      }
      const int i = at + __ffs(kids) - 1;
      at = i + 1;
      double w = positive(sm.p[i]);
      if (a.draft) {
        if (rejected) w = fmax(fma(-c, by_bits(sm.q[i]), w), 0.0);
      } else {
        bool again = false;
        for (int k = lane; k < rejected; k += 32) again |= sm.gone[k] == sm.token[i];
        if (__any_sync(0xffffffffu, again)) w = 0.0;
      }
      if ((double)sm.u[i] * (double)sm.q[i] * Z < w) {
        cur = i;
        ++taken;
        if (rank == 0 && lane == 0) a.path[r * a.path_pitch + taken] = i;
        rejected = 0;
        Z = 1.0;
        c = 0.0;
        summed = false;
      } else if (a.draft) {
        ++rejected;
        c += Z;
        return true;
      } else {
        if (lane == 0) sm.gone[rejected] = sm.token[i];
        __syncwarp();
        ++rejected;
        Z = fmax(Z - w, 0.0);
      }
    }
    return !summed;
  };
  // the decision for the CTA
  auto publish = [&](int done) {
    if (lane == 0) {
      sm.done = done;
      sm.row = sm.row0 + cur;
      sm.rejected = rejected;
      sm.c = c;
    }
  };
  if (warp == 0) {
    if (rank == 0 && lane == 0) a.path[r * a.path_pitch] = 0;
    walk();                                      // nothing is summed yet: it ends in a pass
    publish(0);
  }
  Row row;
  row.gone = sm.gone;
  row.vocab = a.vocab;
  for (int pass = 0;; ++pass) {
    __syncthreads();                             // the decision is there
    row.rejected = sm.rejected;
    row.c = sm.c;
    row.p = a.target + (size_t)sm.row * a.target_pitch;
    row.q = a.draft ? a.draft + (size_t)sm.row * a.draft_pitch : nullptr;
    row.wide = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15u) == 0;
    if (sm.done) break;
    for (int x = c0 + warp; x < c1; x += kWarps) {
      const double t = chunk_total(row, x, lane);
      if (lane == 0) sm.chunk_sum[x - c0] = t;
    }
    __syncthreads();
    if (warp == 0) {
      double t = 0.0;
      for (int x = lane; x < c1 - c0; x += 32) t += sm.chunk_sum[x];
      t = warp_sum(t);
      if (lane < ctas) cluster.map_shared_rank(&sm, lane)->cta_sum[pass & 1][rank] = t;
    }
    cluster.sync();                              // every rank has the totals (by turns: a slower rank may still read the last)
    if (warp == 0) {
      const double* cta_sum = sm.cta_sum[pass & 1];
      double total = 0.0;
      for (int x = 0; x < ctas; ++x) total += cta_sum[x];
      Z = total;
      summed = true;
      // nothing left of w: the children's weights all went to zero by rounding, so take the row itself
      const bool empty = !(total > 0.0);
      if (empty && rejected > 0) {
        rejected = 0;
        c = 0.0;
        at = n;
        summed = false;
      }
      const bool more = walk();
      if (!more && lane == 0) {
        // the CTA of the first total that passes the threshold, or of the last one with any weight
        const double threshold = (double)sm.u_final * total;
        double before = 0.0;
        sm.owner = -1;                           // a row without any weight: no token
        for (int x = 0; x < ctas; ++x) {
          if (cta_sum[x] > 0.0) {
            sm.owner = x;
            sm.before = before;
            if (before + cta_sum[x] > threshold) break;
          }
          before += cta_sum[x];
        }
        sm.threshold = threshold;
      }
      publish(!more);
    }
  }
  if (rank == 0 && tid == 0) {
    a.accept_len[r] = taken;
    if (sm.owner < 0) a.next_token[r] = -1;
  }
  if (rank == sm.owner && warp == 0) {
    // the first chunk that passes the threshold, or the last one with any weight
    const double threshold = sm.threshold;
    double before = sm.before, best_before = before;
    int best = -1;
    for (int x0 = 0; x0 < c1 - c0; x0 += 32) {
      const double t = x0 + lane < c1 - c0 ? sm.chunk_sum[x0 + lane] : 0.0;
      const double incl = warp_scan(t, lane);
      const unsigned past = __ballot_sync(0xffffffffu, t > 0.0 && before + incl > threshold);
      const unsigned any = __ballot_sync(0xffffffffu, t > 0.0);
      if (any) {
        const int where = past ? __ffs(past) - 1 : 31 - __clz(any);
        best = x0 + where;
        best_before = before + __shfl_sync(0xffffffffu, incl - t, where);
      }
      if (past) break;
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int token = best >= 0 ? find_in_chunk(row, c0 + best, best_before, threshold, lane) : -1;
    if (lane == 0) a.next_token[r] = token;
  }
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyLaunch& a, cudaStream_t s) {
  // CTAs a request: up to four an SM in all (two are resident: requests end at different times), and
  // work for half of a CTA's warps.  Trees of 8-32 nodes over 128k tokens with draft rows, up to 2 / 4 / 8 an SM:
  // 64 requests 57 / 53 / 53 us, 75 88 / 74 / 68, 148 98 / 92 / 102, 200 145 / 102 / 94.  Without draft rows, where
  // there is one pass and no chain, two an SM would be ahead: 64 requests 23 / 29 / 31, 148 31 / 47 / 59.
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int chunks = (a.vocab + kChunk - 1) / kChunk;
  int ctas = kMaxCluster;
  while (ctas > 1 && ((long long)a.batch * ctas > 4 * sms || chunks < ctas * kWarps / 2)) ctas >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel, a);
}

}  // namespace pa
