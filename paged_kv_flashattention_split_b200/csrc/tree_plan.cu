// tree_plan.cu - the plan of a draft-tree attention: query tiles, their flat partition, visibility rows.
//
// Request r brings n_r tree nodes whose K/V rows sit behind its cached prefix of p_r = L_r - n_r
// keys; parent[] gives each node's parent.  The plan
//   - cuts the nodes of each request into query tiles of 256 (node, query head) rows of one KV
//     head, 256 / G nodes a tile (G = Hq / Hkv), and the keys into tiles of 128;
//   - lays the units (query tile, key tile) of all requests end to end and gives each of the C
//     CTA slots an equal run of `per` of them, cut into items at the query tiles' borders;
//   - lists the query tiles that were cut, for the merge of their pieces;
//   - writes each node's visibility row: bit j is set if node j is the node itself or one of its
//     ancestors, all zero for a node that is not in use.
// Block 0 does the partition (integer, latency-bound: two block-wide scans), the other blocks
// write the visibility rows, one warp per request; a node's walk up its parents runs in shared
// memory, so its cost is the node's depth, not a chain of global loads.
// 64 requests of up to 16 nodes: 4.2-4.4 us, replayed.
#include <algorithm>

#include "kernels.h"
#include "scan.cuh"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;               // for more than kSmallBatch requests
// up to here 256 threads: barriers of 32 warps cost more than they gain (65 requests of up to 16 nodes: 4.6 us against
// 5.0 with 1024).  Towards the border they gain as much and more: 100 requests 5.0 against 5.1, 256 7.4 against 6.2, and
// with up to 64 nodes, whose rows the fewer threads write, 256 requests 17.0 against 9.5.
constexpr int kSmallBatch = 256;

// Length, first row and node count of request r; false (n = 0) if they are out of range.
__device__ bool read_request(const TreePlanLaunch& a, int r, int* L, int* q0, int* n) {
  *L = a.seq_lens[r];
  *q0 = a.cu_seqlens_q[r];
  const long long q1 = a.cu_seqlens_q[r + 1], cnt = q1 - *q0;
  *n = (int)cnt;
  const bool ok = *L >= 0 && *L <= a.max_kv_len && *q0 >= 0 && q1 <= a.max_q_tokens && cnt >= 0 && cnt <= *L &&
                  cnt <= kTreeMaxNodes;
  if (!ok) *n = 0;
  return ok;
}

// A parent is an earlier node of the request, -1 (a root) or -2 (the node is not in use).
__device__ __forceinline__ bool parent_ok(int p, int i) { return p >= -2 && p < i; }

__device__ void write_bits(const TreePlanLaunch& a, int* parents) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int* par = parents + warp * kTreeMaxNodes;
  for (int r = (blockIdx.x - 1) * warps + warp; r < a.batch; r += (gridDim.x - 1) * warps) {
    int L, q0, n;
    read_request(a, r, &L, &q0, &n);
    for (int i = lane; i < n; i += 32) par[i] = a.parent[q0 + i];
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
      uint32_t bits[kTreeWords];
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) bits[w] = 0;
      int j = i;
      while (j >= 0) {
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w) bits[w] |= (j >> 5) == w ? 1u << (j & 31) : 0u;
        const int p = par[j];
        j = parent_ok(p, j) ? p : -2;              // strictly decreasing, so the walk ends
      }
      if (j != -1) {                               // the chain met a node that is not in use
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w) bits[w] = 0;
      }
      uint4* dst = reinterpret_cast<uint4*>(a.ws.tree_bits + (size_t)(q0 + i) * kTreeWords);
      dst[0] = make_uint4(bits[0], bits[1], bits[2], bits[3]);
      dst[1] = make_uint4(bits[4], bits[5], bits[6], bits[7]);
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(TreePlanLaunch a) {
  extern __shared__ int sm[];
  __shared__ int scan_units[33];
  __shared__ long long scan_items[33];
  // the attention call that follows may be scheduled; it waits for this grid before it reads the plan
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (blockIdx.x > 0) {
    write_bits(a, sm);
    return;
  }
  const int tid = threadIdx.x, nt = blockDim.x;
  WsView ws = a.ws;
  PlanHeader* hdr = ws.hdr;
  const int B = a.batch, qt = tree_tile_nodes(a.hq / a.hkv);
  int* s_tiles = sm;            // [B] query tiles of request r
  int* s_ktiles = sm + B;       // [B] key tiles of request r
  int* s_row = sm + 2 * B;      // [B] its first row
  int* item_slot = sm + 3 * B;  // [max_items]
  if (tid == 0) hdr->error_word = 0;               // every new plan starts with a clean error word
  __syncthreads();
  const int per_t = (B + nt - 1) / nt;
  const int r0 = min(B, tid * per_t), r1 = min(B, r0 + per_t);
  int my_units = 0;
  for (int r = r0; r < r1; ++r) {
    int L, q0, n;
    if (!read_request(a, r, &L, &q0, &n)) set_device_error(hdr, PA_ERR_DEVICE_INDEX);
    const int tiles = (n + qt - 1) / qt, ktiles = n > 0 ? (L + kTreeKvTile - 1) / kTreeKvTile : 0;
    s_tiles[r] = tiles;
    s_ktiles[r] = ktiles;
    s_row[r] = q0;
    ws.req_splits[r] = tiles;
    ws.req_len[r] = L;
    ws.req_aux[r] = q0;
    ws.req_prefix[r] = n > 0 ? L - n : L;
    my_units += tiles * ktiles;
  }
  // the parents, checked here so that only this block writes the error word; all loads at once, the scans
  // hide them.  Rows before the first request's belong to something else.  (With offsets out of range the
  // search may find a wrong request: the error is there then.)
  const int rows = max(0, min(a.cu_seqlens_q[B], a.max_q_tokens));
  const int row0 = max(0, min(a.cu_seqlens_q[0], rows)) + tid;
  int parent[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) parent[k] = row0 + k * nt < rows ? a.parent[row0 + k * nt] : -1;
  int total = 0;
  const int units0 = block_exclusive_scan(my_units, scan_units, &total);
  const int per = max(1, (int)(((long long)total + a.slots - 1) / a.slots));
  // items: each query tile's units [g, g + k) cut at the slots' borders; cut tiles in the upper half
  long long mine = 0, all = 0;
  for (int r = r0, g = units0; r < r1; ++r)
    for (int t = 0, k = s_ktiles[r]; t < s_tiles[r]; ++t, g += k) {
      const int pieces = (g + k - 1) / per - g / per + 1;
      mine += pieces + (pieces > 1 ? 1LL << 32 : 0);
    }
  const long long before = block_exclusive_scan(mine, scan_items, &all);
  int n_items = (int)(all & 0xFFFFFFFF), n_cut = (int)(all >> 32);
  if (n_items > a.max_items || n_cut > a.max_cut) {        // rows of Q that requests share: too many of them in all
    if (tid == 0) set_device_error(hdr, PA_ERR_DEVICE_INDEX);
    n_items = min(n_items, a.max_items);
    n_cut = min(n_cut, a.max_cut);
  }
  int i = (int)(before & 0xFFFFFFFF), cut = (int)(before >> 32);
  for (int r = r0, g = units0; r < r1; ++r) {
    ws.req_base[r] = g;
    for (int t = 0, k = s_ktiles[r]; t < s_tiles[r]; ++t, g += k) {
      const int c0 = g / per, c1 = (g + k - 1) / per;
      if (c1 > c0) {
        if (cut < n_cut) ws.tree_tiles[cut] = make_int2(r, t);
        ++cut;
      }
      for (int c = c0; c <= c1; ++c, ++i) {
        if (i >= n_items) break;
        ws.items[i] = make_int4(r, t, (int)(max((long long)g, (long long)c * per) - g),
                                (int)(min((long long)g + k, (long long)(c + 1) * per) - g));
        item_slot[i] = c;
      }
    }
  }
  if (tid == 0) ws.req_base[B] = total;
  auto check = [&](int row, int p) {
    int lo = 0, hi = B;                            // the request of the row: the last one that starts at or before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_row[mid] <= row) lo = mid; else hi = mid;
    }
    if (!parent_ok(p, row - s_row[lo])) set_device_error(hdr, PA_ERR_DEVICE_INDEX);
  };
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (row0 + k * nt < rows) check(row0 + k * nt, parent[k]);
  for (int row = row0 + 4 * nt; row < rows; row += nt) check(row, a.parent[row]);
  __syncthreads();
  // slot_first[c] = first item whose slot is >= c (slots are non-decreasing along the list)
  for (int x = tid; x < n_items; x += nt) {
    const int prev = x > 0 ? item_slot[x - 1] : -1;
    for (int c = prev + 1; c <= item_slot[x]; ++c) ws.slot_first[c] = x;
  }
  for (int c = tid + (n_items > 0 ? item_slot[n_items - 1] + 1 : 0); c <= a.slots; c += nt) ws.slot_first[c] = n_items;
  if (tid == 0) {
    hdr->magic = kMagic;
    hdr->mode = PA_MODE_TREE;
    hdr->batch = B;
    hdr->hq = a.hq;
    hdr->hkv = a.hkv;
    hdr->head_dim = a.head_dim;
    hdr->page_size = a.page_size;
    hdr->num_items = n_items;
    hdr->max_items = a.max_items;
    hdr->tile = kTreeKvTile;
    hdr->chunk_tiles = per;
    hdr->num_sms = a.num_sms;
    hdr->max_splits = 0;
    hdr->slots = a.slots;
    hdr->reserved1 = n_cut;
  }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanLaunch& a, cudaStream_t s) {
  const int threads = a.batch <= kSmallBatch ? 256 : kPlanThreads, warps = threads / 32;
  const size_t smem = std::max(sizeof(int) * (3 * (size_t)a.batch + (size_t)a.max_items),
                               sizeof(int) * warps * kTreeMaxNodes);
  constexpr int kSmemMax = (int)(sizeof(int) * (3 * (size_t)kMaxBatch + kMaxSortItems));
  static std::atomic<bool> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(tree_plan_kernel, kSmemMax, smem_set);
  if (e != cudaSuccess) return e;
  tree_plan_kernel<<<1 + (a.batch + warps - 1) / warps, threads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
