// Eviction from a key/value cache by accumulated attention weight, and the
// commit of accepted drafts (the same update with room for every candidate).
//
// Each (sequence, kv head) keeps the m candidates that rank first by (held,
// weight descending, slot ascending). The rank is a 32-bit key whose unsigned
// order is that of the weights; held slots take the largest key, slots that
// are no candidates the key 0. The m-th largest key is found by a radix
// search (digits of 11, 11 and 10 bits from the top, one histogram each);
// among equal keys the first slots win.
//
// The kept rows must end in slots 0 .. m-1, and the order of slots carries no
// meaning, so only as many rows move as there are unkept slots below m: the
// i-th such hole takes the i-th kept row from m on. Sources lie at m or
// above and destinations below, so the moves commute and need no order.
//
// One thread-block cluster per (sequence, head): its blocks split the slots,
// hold the keys in shared memory, and read each other's histograms and
// counts through distributed shared memory, so the whole update is one
// launch. Bound: 8 bytes (weight, position) per slot and 1 KB per moved row
// against HBM; for small caches the chain of three histogram rounds, two
// count rounds and their cluster barriers.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace cg = cooperative_groups;

namespace dhsa {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;
constexpr int kRounds = 3;
constexpr int kMaxCluster = 8;            // portable cluster size
constexpr int kKeysPerBlock = 48 * 1024;  // keys held in shared memory; later ones are derived again
constexpr int kSlotsPerBlock = 8192;      // slots a block of a cluster is given before another one joins

struct EvictParams {
  __nv_bfloat16 *K, *V;
  RowStrides ks, vs;
  const float* weight;
  const int32_t* pos;
  const int32_t *lengths, *n_draft, *next_pos;
  const int64_t* accept;
  float* weight_out;
  int32_t *pos_out, *lengths_out, *index;
  int32_t* lists;          // [B * Hkv][cap]: holes in the first half, their sources in the second
  int B, Hkv, cap, keep, sinks, recent, index_cols, max_draft, keys_held;
  unsigned int* status;
};

// unsigned order = order of the floats, NaN lowest, -0 equal to +0; at least 1
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
  uint32_t hist[kRounds][kBins];
  uint32_t warp_sum[kEvWarps];
  uint32_t warp_a[kEvWarps], warp_b[kEvWarps];
  uint32_t pick_bin, pick_above;
  uint32_t total[3];         // this block's ties, holes, sources (read by the cluster)
};

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char ev_smem[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(ev_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + sizeof(EvictShared));
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / C;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const SeqLen sl = seq_len(p.lengths, p.n_draft, 0, b, p.max_draft, p.cap);
  uint64_t bits = p.accept ? (uint64_t)p.accept[b] : ~0ull;
  bits &= sl.draft >= 64 ? ~0ull : (1ull << sl.draft) - 1;
  const int n_cand = sl.len + __popcll(bits), n_all = sl.len + sl.draft;
  const int m = min(p.keep, n_cand);
  if (sl.bad && rank == 0 && tid == 0) raise_device_flag(p.status, DHSA_DEVFLAG_BAD_CACHE);
  if (rank == 0 && h == 0 && tid == 0) p.lengths_out[b] = m;

  const long long row = (long long)bh * p.cap;
  const float* w_in = p.weight + row;
  const int32_t* pos_in = p.pos + row;
  const long long held_from = p.next_pos ? (long long)p.next_pos[b] - p.recent : (long long)INT32_MAX + 1;

  // this block's slots, and each warp's contiguous share of them
  const int per_warp = ceil_div(ceil_div(n_all, C * kEvWarps), 32) * 32;
  const int blk0 = rank * per_warp * kEvWarps;
  const int w0 = blk0 + warp * per_warp, w1 = min(w0 + per_warp, n_all);

  auto is_cand = [&](int s) { return s < sl.len || ((bits >> (s - sl.len)) & 1ull); };
  auto make_key = [&](int s) -> uint32_t {
    if (!is_cand(s)) return 0u;
    const int q = pos_in[s];
    return (q < p.sinks || q >= held_from) ? 0xFFFFFFFFu : weight_key(w_in[s]);
  };

  const bool all = m == n_cand;            // every candidate stays: no ranking
  uint32_t cut = 0;                        // the m-th largest key
  uint32_t ties = 0;                       // how many of the slots with that key stay
  if (!all) {
    for (int i = tid; i < kRounds * kBins; i += kEvThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    for (int s = w0 + lane; s < w1; s += 32) {
      const uint32_t k = make_key(s);
      if (s - blk0 < p.keys_held) keys[s - blk0] = k;
      atomicAdd(&sh.hist[0][k >> 21], 1u);
    }
  }
  auto key_of = [&](int s) { return s - blk0 < p.keys_held ? keys[s - blk0] : make_key(s); };

  if (!all) {
    uint32_t left = (uint32_t)m;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int shift = r == 0 ? 21 : r == 1 ? 10 : 0;
      if (r > 0) {
        const int above = r == 1 ? 21 : 10;
        const uint32_t mask = r == 1 ? 0x7FFu : 0x3FFu;
        for (int s = w0 + lane; s < w1; s += 32) {
          const uint32_t k = key_of(s);
          if ((k >> above) == (cut >> above)) atomicAdd(&sh.hist[r][(k >> shift) & mask], 1u);
        }
      }
      cluster.sync();
      // suffix sums from the top bin: thread t holds bins 2047-2t and 2046-2t
      uint32_t c0 = 0, c1 = 0;
      const int hi = kBins - 1 - 2 * tid;
      for (int c = 0; c < C; ++c) {
        const uint32_t* rh = cluster.map_shared_rank(&sh.hist[r][0], c);
        c0 += rh[hi];
        c1 += rh[hi - 1];
      }
      uint32_t inc = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      __syncthreads();
      uint32_t before = inc - (c0 + c1);
      for (int i = 0; i < warp; ++i) before += sh.warp_sum[i];
      // exactly one bin holds the left-th key from the top
      if (before < left && left <= before + c0) {
        sh.pick_bin = hi;
        sh.pick_above = before;
      } else if (before + c0 < left && left <= before + c0 + c1) {
        sh.pick_bin = hi - 1;
        sh.pick_above = before + c0;
      }
      __syncthreads();
      cut |= sh.pick_bin << shift;
      left -= sh.pick_above;
      __syncthreads();
    }
    ties = left;
  }

  // an exclusive sum over the cluster's blocks and this block's warps
  auto warp_offsets = [&](uint32_t* sums, int which) {
    __syncthreads();
    if (tid == 0) {
      uint32_t t = 0;
      for (int i = 0; i < kEvWarps; ++i) t += sums[i];
      sh.total[which] = t;
    }
  };
  auto below = [&](const uint32_t* sums, int which) {
    uint32_t t = 0;
    for (int c = 0; c < rank; ++c) t += *cluster.map_shared_rank(&sh.total[which], c);
    for (int i = 0; i < warp; ++i) t += sums[i];
    return t;
  };

  uint32_t tie_at = 0;
  if (!all) {
    uint32_t n = 0;
    for (int s0 = w0; s0 < w1; s0 += 32) {
      const int s = s0 + lane;
      n += __popc(__ballot_sync(0xffffffffu, s < w1 && key_of(s) == cut));
    }
    if (lane == 0) sh.warp_sum[warp] = n;
    warp_offsets(sh.warp_sum, 0);
    cluster.sync();
    tie_at = below(sh.warp_sum, 0);
  }
  const uint32_t lt = (1u << lane) - 1;
  // whether slot s stays; called for 32 consecutive slots by a whole warp, in
  // order, with the running count of equal keys before them
  auto stays = [&](int s, uint32_t& tie_run) {
    if (all) return s < w1 && is_cand(s);
    const uint32_t k = s < w1 ? key_of(s) : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, s < w1 && k == cut);
    const bool yes = s < w1 && (k > cut || (k == cut && tie_run + __popc(eq & lt) < ties));
    tie_run += __popc(eq);
    return yes;
  };

  uint32_t tie_run = tie_at, holes = 0, srcs = 0;
  for (int s0 = w0; s0 < w1; s0 += 32) {
    const int s = s0 + lane;
    const bool yes = stays(s, tie_run);
    holes += __popc(__ballot_sync(0xffffffffu, s < m && s < w1 && !yes));
    srcs += __popc(__ballot_sync(0xffffffffu, s >= m && yes));
  }
  if (lane == 0) {
    sh.warp_a[warp] = holes;
    sh.warp_b[warp] = srcs;
  }
  warp_offsets(sh.warp_a, 1);
  warp_offsets(sh.warp_b, 2);
  cluster.sync();
  uint32_t hole_at = below(sh.warp_a, 1), src_at = below(sh.warp_b, 2);

  // the lists, and what stays where it is
  int32_t* hole_list = p.lists + row;
  int32_t* src_list = hole_list + p.cap / 2;   // min(m, n_all - m) <= cap / 2 rows move
  int32_t* idx_row = p.index ? p.index + (long long)bh * p.index_cols : nullptr;
  float* w_out = p.weight_out + row;
  int32_t* pos_out = p.pos_out + row;
  tie_run = tie_at;
  for (int s0 = w0; s0 < w1; s0 += 32) {
    const int s = s0 + lane;
    const bool yes = stays(s, tie_run);
    const bool hole = s < m && s < w1 && !yes, src = s >= m && yes;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), sb = __ballot_sync(0xffffffffu, src);
    if (hole) hole_list[hole_at + __popc(hb & lt)] = s;
    if (src) src_list[src_at + __popc(sb & lt)] = s;
    hole_at += __popc(hb);
    src_at += __popc(sb);
    if (yes && s < m) {
      if (idx_row) idx_row[s] = s;
      if (w_out != w_in) w_out[s] = w_in[s];
      if (pos_out != pos_in) pos_out[s] = pos_in[s];
    }
  }
  if (idx_row)
    for (int s = m + rank * kEvThreads + tid; s < p.index_cols; s += C * kEvThreads) idx_row[s] = -1;
  // the cluster's lists are complete, and nobody reads a weight or position
  // to rank it any more
  cluster.sync();
  uint32_t moves = 0;
  for (int c = 0; c < C; ++c) moves += *cluster.map_shared_rank(&sh.total[1], c);
  // one warp per moved slot: 16 lanes carry its K row, 16 its V row
  const bool is_v = lane >= 16;
  __nv_bfloat16* base = is_v ? p.V + b * p.vs.b + h * p.vs.h : p.K + b * p.ks.b + h * p.ks.h;
  const long long rs = is_v ? p.vs.r : p.ks.r;
  base += (lane & 15) * 8;
  constexpr int kInFlight = 4;
  const int stride = C * kEvWarps;
  for (uint32_t r0 = rank * kEvWarps + warp; r0 < moves; r0 += kInFlight * stride) {
    uint4 x[kInFlight];
    int dst[kInFlight], from[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const uint32_t r = r0 + k * stride;
      dst[k] = -1;
      if (r < moves) {
        dst[k] = hole_list[r];
        from[k] = src_list[r];
        x[k] = *reinterpret_cast<const uint4*>(base + from[k] * rs);
      }
    }
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (dst[k] < 0) continue;
      *reinterpret_cast<uint4*>(base + dst[k] * rs) = x[k];
      if (lane == 0) {
        w_out[dst[k]] = w_in[from[k]];
        if (idx_row) idx_row[dst[k]] = from[k];
      }
      if (lane == 16) pos_out[dst[k]] = pos_in[from[k]];
    }
  }
  // no block leaves while another may still read its counts
  cluster.sync();
}

int cluster_size(int cap) {
  int c = 1;
  while (c < kMaxCluster && (long long)c * kSlotsPerBlock < cap) c *= 2;
  return c;
}

}  // namespace

size_t evict_ws_bytes(int B, int Hkv, int cap) { return sizeof(int32_t) * (size_t)B * Hkv * cap; }
int evict_max_drafts() { return 64; }

int launch_evict(void* K, const RowStrides& ks, void* V, const RowStrides& vs, const float* weight,
                 const int32_t* pos, int B, int Hkv, int cap, const int32_t* lengths, const int32_t* n_draft,
                 const int64_t* accept, int keep, int sinks, int recent, const int32_t* next_pos, float* weight_out,
                 int32_t* pos_out, int32_t* lengths_out, int32_t* index, void* ws, unsigned int* status,
                 cudaStream_t stream) {
  EvictParams p;
  p.K = static_cast<__nv_bfloat16*>(K);
  p.V = static_cast<__nv_bfloat16*>(V);
  p.ks = ks;
  p.vs = vs;
  p.weight = weight;
  p.pos = pos;
  p.lengths = lengths;
  p.n_draft = n_draft;
  p.next_pos = next_pos;
  p.accept = accept;
  p.weight_out = weight_out;
  p.pos_out = pos_out;
  p.lengths_out = lengths_out;
  p.index = index;
  p.lists = static_cast<int32_t*>(ws);
  p.B = B;
  p.Hkv = Hkv;
  p.cap = cap;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.index_cols = keep < cap ? keep : cap;
  p.max_draft = evict_max_drafts();
  p.status = status;
  const int C = cluster_size(cap);
  const int span = ceil_div(ceil_div(cap, C * kEvWarps), 32) * 32 * kEvWarps;   // slots of one block at most
  p.keys_held = span < kKeysPerBlock ? span : kKeysPerBlock;
  const size_t smem = sizeof(EvictShared) + 4u * (size_t)p.keys_held;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(EvictShared) + 4u * (size_t)kKeysPerBlock));
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * Hkv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, evict_kernel, p));
}

}  // namespace dhsa
